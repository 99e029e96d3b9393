"""Gradients of attention with modified scores where those of some samples or tokens are far smaller than
others' (losses that mask or weight tokens), against the fp64 oracle (bounds: scored_util), and the choice
between f16 and bf16 operands that each sample's own range makes."""
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


def _gradients(x, cu, scale, **opt):
    from vlm_zigzag_head_gb300 import ScorePlan, cp_attn_scored_bwd, cp_attn_scored_fwd
    x = [t.to(DEV) for t in x]
    plan = ScorePlan(cu, x[0].shape[1], rel_buckets=[0, 1, 2], device=DEV)
    out, lse, lo = cp_attn_scored_fwd(*x[:3], plan, scale, residual=True, **opt)
    return [O._f64(t) for t in cp_attn_scored_bwd(*x[:3], out, lse, x[3], plan, scale, out_lo=lo, **opt)]


def _random(T, H, Hkv, d, seed, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    x = [torch.randn((T, h, d), generator=g) for h in (H, Hkv, Hkv, H)]
    x[0] *= gain
    return [t.to(torch.bfloat16) for t in x]


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[1024], [513, 130, 90], [200, 1500]])
@pytest.mark.parametrize("cap", [0.0, 5.0])
@pytest.mark.parametrize("d", [64, 128])
def test_short_samples_of_even_gradients_have_f16_operands(lens, cap, d):
    """At softmax scale 1 the forward's probabilities are f16 too, so that P, D and dS are off by half a step
    of f16 at most, 2^-11, whose rms is below a quarter of that: 2^-10 in norm leaves room for their sums.
    bf16 dS is off by 1.6e-3 in norm, as in the long sample beside."""
    cu = [0] + [int(n) for n in np.cumsum(lens)]
    x = _random(cu[-1], 4, 2, d, d, d ** -0.5)
    got = _gradients(x, cu, 1.0, softcap=cap)
    want = O.scored_attention(*x[:3], cu, 1.0, O.Scores(softcap=cap), x[3])[2:5]
    for name, a, b in zip(("dq", "dk"), got, want):
        for i, n in enumerate(lens):
            rows = slice(cu[i], cu[i + 1])
            err = np.linalg.norm(a[rows] - b[rows]) / np.linalg.norm(b[rows])
            assert err <= 2.0 ** -10 if n <= 1024 else 2.0 ** -10 < err <= 2.0 ** -8, (name, n, err)


@pytest.mark.gpu
@pytest.mark.parametrize("beside", [[1025], [1024], [40, 3000], [1]])
@pytest.mark.parametrize("kind", list(OPTIONS))
def test_a_sample_does_not_notice_the_lengths_of_others(beside, kind):
    """Backward from the same forward results.  (The forward's runs are cut by the whole packing; a part
    rounds its probabilities relative to its own maximum, so out and D differ by roundings of P.)"""
    from vlm_zigzag_head_gb300 import ScorePlan, cp_attn_scored_bwd, cp_attn_scored_fwd
    n, H, d = 300, 4, 64
    cu = [0, n] + [n + int(m) for m in np.cumsum(beside)]
    x = _random(cu[-1], H, 1, d, 9)
    opt = dict(OPTIONS[kind])
    if "slopes" in opt:
        opt["slopes"] = torch.tensor([0.5, 0.03, 0.1, 0.2], device=DEV)
    if opt.pop("bias", False):
        opt["rel_bias"] = torch.randn(H, 3, device=DEV, generator=torch.Generator(DEV).manual_seed(1))
    x = [t.to(DEV) for t in x]
    alone, rest, whole = (ScorePlan(c, H, rel_buckets=[0, 1, 2], device=DEV)
                          for c in (cu[:2], [m - n for m in cu[1:]], cu))
    a = cp_attn_scored_fwd(*(t[:n] for t in x[:3]), alone, 0.125, residual=True, **opt)
    b = cp_attn_scored_fwd(*(t[n:] for t in x[:3]), rest, 0.125, residual=True, **opt)
    both = [torch.cat(t, dim=i) for i, t in zip((0, 1, 0), zip(a, b))]
    want = cp_attn_scored_bwd(*(t[:n] for t in x[:3]), *a[:2], x[3][:n], alone, 0.125, out_lo=a[2], **opt)
    got = cp_attn_scored_bwd(*x[:3], *both[:2], x[3], whole, 0.125, out_lo=both[2], **opt)
    for name, s, t in zip(("dq", "dk", "dv"), got, want):
        assert (s[:n] - t).norm() <= 1e-5 * t.norm(), name   # the order of fp32 sums


@pytest.mark.gpu
@pytest.mark.parametrize("power", [-100, -45, -20, -8, 12, 45, 90])
def test_gradients_are_linear_in_dout(power):
    """dout times a power of two: within the range of the f16 scales the operands have the same bits, up to the
    order of fp32 sums; far outside it they are bf16, within its bound."""
    cu, d = [0, 300, 400], 64
    x = _random(cu[-1], 2, 1, d, 4)
    want = _gradients(x, cu, 0.125, softcap=5.0)
    y = x[:3] + [(x[3].float() * 2.0 ** power).to(torch.bfloat16)]
    got = _gradients(y, cu, 0.125, softcap=5.0)
    if abs(power) <= 45:
        for a, b in zip(got, want):
            assert np.linalg.norm(a * 2.0 ** -power - b) <= 1e-5 * np.linalg.norm(b)
    vals, tol = reference(*y[:3], cu, 0.125, O.Scores(softcap=5.0), y[3], BF16, BF16)
    for name, a in zip(("dq", "dk", "dv"), got):
        check(name, a, vals[name], tol[name])


@pytest.mark.gpu
@pytest.mark.parametrize("ratio", [2.0 ** -7, 2.0 ** -9])
@pytest.mark.parametrize("grow", [1.0, 1e4])
def test_rows_on_both_sides_of_the_ratio_that_f16_takes(ratio, grow):
    """Every third row's dout is 2^-7 (f16) or 2^-9 (bf16) of the rest's, the last 20 rows' is zero; q and v
    of the next sample are 1e4 times as large."""
    cu, d = [0, 500, 620], 128
    x = _random(cu[-1], 2, 2, d, 6)
    at = torch.arange(cu[-1])
    f = torch.where((at % 3 == 0) & (at < 500), ratio, 1.0) * ((at < 480) | (at >= 500)).float()
    x[3] = (x[3].float() * f[:, None, None]).to(torch.bfloat16)
    for t in (x[0], x[2]):
        t[500:] *= grow
    got = _gradients(x, cu, d ** -0.5)
    vals, tol = reference(*x[:3], cu, d ** -0.5, O.Scores(), x[3], BF16, BF16)
    for name, a in zip(("dq", "dk", "dv"), got):
        check(name, a, vals[name], tol[name])
    assert not got[0][480:500].any()
