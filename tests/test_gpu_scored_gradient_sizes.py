"""Gradients of attention with modified scores where those of some samples or tokens are far smaller than
others' (losses that mask or weight tokens), against the fp64 oracle (bounds: scored_util)."""
import numpy as np
import pytest
import torch

from oracle import scored as O
from scored_util import check, reference

DEV = "cuda:0"
BF16 = 2.0 ** -8
OPTIONS = {"plain": {}, "cap": dict(softcap=5.0), "slopes": dict(slopes=[0.5, 0.03]), "bias": dict(bias=True),
           "cap_bias": dict(softcap=5.0, bias=True)}


@pytest.mark.gpu
@pytest.mark.parametrize("where", ["sample", "tokens"])
@pytest.mark.parametrize("kind", list(OPTIONS))
@pytest.mark.parametrize("d,scale,small", [(64, 0.125, 1e-6), (128, 128 ** -0.5, 1e-8), (64, 1.0, 1e-6)])
def test_small_gradients_keep_their_precision(d, scale, small, kind, where):
    """A sample's dout (or that of every other 50 tokens) is 1e-6 or 1e-8 of the rest's: its dq, and in the
    sample dk and dv, are as exact as any.  The bounds follow each row's own dout."""
    from vlm_zigzag_head_gb300 import ScorePlan, cp_attn_scored_bwd, cp_attn_scored_fwd, relative_buckets
    cu, H = [0, 300, 812], 2
    g = torch.Generator().manual_seed(d)
    gain = 1.0 if scale < 0.5 else d ** -0.5
    q, k, v, dout = (torch.randn((cu[-1], h, d), generator=g) for h in (H, 1, 1, H))
    at = torch.arange(cu[-1])
    dout *= torch.where(at < 300 if where == "sample" else at // 50 % 2 == 0, small, 1.0)[:, None, None]
    q, k, v, dout = (x.to(torch.bfloat16) for x in (q * gain, k, v, dout))
    opt = dict(OPTIONS[kind])
    slopes = torch.tensor(opt["slopes"]) if "slopes" in opt else None
    bias = torch.randn((H, 8), generator=g) if "bias" in opt else None
    buckets = relative_buckets(8, 32)
    cap = opt.get("softcap", 0.0)
    plan = ScorePlan(cu, H, rel_buckets=buckets, device=DEV)
    x = [t.to(DEV) for t in (q, k, v, dout)]
    extra = dict(softcap=cap, slopes=None if slopes is None else slopes.to(DEV),
                 rel_bias=None if bias is None else bias.to(DEV))
    out, lse, lo = cp_attn_scored_fwd(*x[:3], plan, scale, residual=True, **extra)
    got = cp_attn_scored_bwd(*x[:3], out, lse, x[3], plan, scale, out_lo=lo, **extra)
    s = O.Scores(softcap=cap, slopes=slopes, bias=bias, buckets=buckets)
    vals, tol = reference(q, k, v, cu, scale, s, dout, BF16, BF16)
    for name, a in zip(("dq", "dk", "dv", "dbias"), got):
        check(name, a, vals[name], tol[name])


@pytest.mark.gpu
@pytest.mark.parametrize("kind", list(OPTIONS))
def test_a_sample_gets_the_gradients_it_gets_alone(kind):
    """Beside a sample whose dout is 1e6 times as large, and whose v has an outlier."""
    from vlm_zigzag_head_gb300 import ScorePlan, cp_attn_scored_bwd, cp_attn_scored_fwd
    H, d, n = 2, 64, 256
    g = torch.Generator().manual_seed(3)
    q, k, v, dout = (torch.randn((2 * n, h, d), generator=g) for h in (H, 1, 1, H))
    dout[n:] *= 1e6
    v[n + 5] *= 1e3
    x = [t.to(torch.bfloat16).to(DEV) for t in (q, k, v, dout)]
    opt = dict(OPTIONS[kind])
    if "slopes" in opt:
        opt["slopes"] = torch.tensor(opt["slopes"], device=DEV)
    if opt.pop("bias", False):
        opt["rel_bias"] = torch.randn((H, 3), generator=g).to(DEV)
    ends = []
    for cu in ([0, n, 2 * n], [0, n]):
        plan = ScorePlan(cu, H, rel_buckets=[0, 1, 2], device=DEV)
        y = [t[:cu[-1]].contiguous() for t in x]
        out, lse, lo = cp_attn_scored_fwd(*y[:3], plan, 0.125, residual=True, **opt)
        ends.append(cp_attn_scored_bwd(*y[:3], out, lse, y[3], plan, 0.125, out_lo=lo, **opt)[:3])
    for name, a, b in zip(("dq", "dk", "dv"), *ends):
        a, b = (O._f64(t[:n]) for t in (a, b))
        # equal up to the order of fp32 sums; a bias's V in f16 with another power of two is exact here
        assert np.linalg.norm(a - b) <= 1e-5 * np.linalg.norm(b), name
