"""Attention with modified scores against the fp64 oracle (bounds: scored_util)."""
import numpy as np
import pytest
import torch

from oracle import scored as O
from scored_util import check, f16_ds_floor, reference

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def _cu(lens):
    return [0] + [int(x) for x in np.cumsum(lens)]


def _inputs(T, H, Hkv, d, dtype, seed, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    q, dout = (torch.randn((T, H, d), generator=g) for _ in range(2))
    k, v = (torch.randn((T, Hkv, d), generator=g) for _ in range(2))
    return [(x * f).to(DT[dtype]) for x, f in ((q, gain), (k, 1.0), (v, 1.0), (dout, 1.0))]


def _bias(H, kind, seed, dtype=torch.float32):
    """(slopes, rel_bias, buckets) of a case's bias: None, "slopes" or (n_buckets, max_distance)."""
    from vlm_zigzag_head_gb300 import relative_buckets
    g = torch.Generator().manual_seed(seed)
    if kind is None:
        return None, None, None
    if kind == "slopes":
        return torch.tensor([2.0 ** (-1 - h % 8) for h in range(H)]), None, None
    return None, torch.randn((H, kind[0]), generator=g).to(dtype), relative_buckets(*kind)


def _run(lens, prefix, both, H, Hkv, d, dtype, scale, cap, kind, gain=1.0, bias_dtype=torch.float32, seed=0):
    from vlm_zigzag_head_gb300 import ScorePlan, Workspace, cp_attn_scored_bwd, cp_attn_scored_fwd, cp_workspace_status
    cu = _cu(lens)
    q, k, v, dout = _inputs(cu[-1], H, Hkv, d, dtype, seed, gain)
    slopes, bias, buckets = _bias(H, kind, seed + 1, bias_dtype)
    plan = ScorePlan(cu, H, prefix_len=prefix, bidirectional_prefix=both, rel_buckets=buckets, device=DEV)
    dv = [x.to(DEV) for x in (q, k, v, dout)]
    extra = dict(softcap=cap, slopes=None if slopes is None else slopes.to(DEV),
                 rel_bias=None if bias is None else bias.to(DEV))
    ws = Workspace(DEV)
    out, lse, *lo = cp_attn_scored_fwd(*dv[:3], plan, scale, residual=dtype == "bf16", workspace=ws, **extra)
    assert cp_workspace_status(ws) == 0
    got = cp_attn_scored_bwd(*dv[:3], out, lse, dv[3], plan, scale, workspace=ws, out_lo=lo[0] if lo else None,
                             **extra)
    assert cp_workspace_status(ws) == 0
    pre = [prefix] * len(lens) if isinstance(prefix, int) else prefix
    s = O.Scores(softcap=cap, slopes=slopes, bias=bias, buckets=buckets, prefix_lens=pre, bidirectional=both)
    vals, tol = reference(q, k, v, cu, scale, s, dout, HALF_STEP[dtype] if dtype == "bf16" else 0.0,
                          HALF_STEP[dtype], f16_ds_floor(v, dout) if dtype == "bf16" else 0.0)
    check("out", out, vals["out"], tol["out"])
    check("lse", lse, vals["lse"], tol["lse"])
    for name, g in zip(("dq", "dk", "dv", "dbias"), got):
        check(name, g, vals[name], tol[name])


R128, R64 = 128 ** -0.5, 0.125
CASES = [   # lens, prefix, both, H, Hkv, d, scale, cap, bias
    ([1], 0, False, 1, 1, 64, R64, 0.0, "slopes"),
    ([1], 1, True, 2, 1, 128, R128, 5.0, None),
    ([128], 0, False, 2, 2, 128, R128, 30.0, None),
    ([129, 0, 255], 0, False, 2, 1, 64, R64, 30.0, None),
    ([257, 1, 2], 0, False, 4, 1, 128, R128, 0.0, "slopes"),
    ([300, 77], [100, 77], True, 3, 1, 128, R128, 0.0, None),
    ([300, 401], [129, 1], True, 6, 2, 64, R64, 0.0, "slopes"),
    ([520], 256, True, 2, 2, 128, R128, 20.0, "slopes"),
    ([520, 130], 130, True, 6, 1, 64, R64, 20.0, "slopes"),
    ([385], 0, False, 2, 2, 64, R64, 0.0, (8, 16)),
    ([640, 31], 0, False, 4, 2, 128, R128, 0.0, (32, 128)),
    ([700], 200, True, 2, 1, 64, R64, 0.0, (16, 600)),
    ([333, 200], 150, True, 4, 1, 128, R128, 10.0, (32, 64)),
    ([200], 0, False, 2, 2, 64, 1.0, 0.0, (32, 128)),       # scale 1: f16 operands
    ([260, 130], 60, True, 4, 2, 128, 1.0, 0.0, "slopes"),
    ([260], 0, False, 2, 1, 64, 1.0, 4.0, None),
    ([260], 40, True, 2, 1, 128, 1.0, 4.0, (8, 32)),
    ([40] * 20, 3, True, 32, 32, 64, R64, 8.0, "slopes"),     # more units than four per SM
]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,prefix,both,H,Hkv,d,scale,cap,kind", CASES)
def test_bf16_matches_oracle(lens, prefix, both, H, Hkv, d, scale, cap, kind):
    gain = 1.0 if scale < 0.5 else d ** -0.5     # queries that carry the scaling
    _run(lens, prefix, both, H, Hkv, d, "bf16", scale, cap, kind, gain, seed=len(lens) + d)


@pytest.mark.gpu
@pytest.mark.parametrize("cap,gain", [(2.0, 1.0), (1.0, 6.0), (0.01, 1.0), (6.0, 2.0)])
@pytest.mark.parametrize("kind", [None, "slopes", (8, 32)])
def test_bf16_saturated_caps(cap, gain, kind):
    """Scores far beyond the cap, and tiles on both sides of the polynomial's range."""
    _run([270], 0, False, 2, 1, 64, "bf16", R64, cap, kind, gain, seed=3)


F32 = [([1], 0, False, 1, 1, 64, R64, 0.0, None), ([64, 65], 0, False, 2, 1, 64, R64, 10.0, None),
       ([130, 0, 3], [70, 0, 3], True, 4, 2, 128, R128, 0.0, "slopes"),
       ([200], 0, False, 3, 1, 64, 1.0, 0.0, (8, 32)), ([190, 20], [90, 20], True, 2, 2, 128, R128, 3.0, (32, 128)),
       ([129], 129, True, 2, 2, 64, R64, 20.0, "slopes")]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,prefix,both,H,Hkv,d,scale,cap,kind", F32)
def test_f32_matches_oracle(lens, prefix, both, H, Hkv, d, scale, cap, kind):
    gain = 1.0 if scale < 0.5 else d ** -0.5
    _run(lens, prefix, both, H, Hkv, d, "f32", scale, cap, kind, gain, seed=d)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hide", [float("-inf"), torch.finfo(torch.float32).min, -1e37])
def test_bias_that_hides_keys(dtype, hide):
    """Hidden distances leave some rows, or all, without a key: out 0, lse -inf, no gradient."""
    from vlm_zigzag_head_gb300 import ScorePlan, cp_attn_scored_bwd, cp_attn_scored_fwd
    H, d, cu, buckets = 4, 64, [0, 140, 150], [0, 1, 2]
    bias = torch.zeros(H, 3)
    bias[0, :] = hide               # nothing left
    bias[1, 0] = hide               # not itself: the first row is empty
    bias[2, 2] = hide               # itself and its neighbour
    bias[3, 1] = 0.5
    q, k, v, dout = _inputs(cu[-1], H, 2, d, dtype, 5)
    plan = ScorePlan(cu, H, rel_buckets=buckets, device=DEV)
    dv = [x.to(DEV) for x in (q, k, v, dout)]
    out, lse, *lo = cp_attn_scored_fwd(*dv[:3], plan, R64, rel_bias=bias.to(DEV), residual=dtype == "bf16")
    got = cp_attn_scored_bwd(*dv[:3], out, lse, dv[3], plan, R64, rel_bias=bias.to(DEV),
                             out_lo=lo[0] if lo else None)
    s = O.Scores(bias=bias.clamp(min=-1e38), buckets=buckets)
    vals, tol = reference(q, k, v, cu, R64, s, dout, HALF_STEP[dtype] if dtype == "bf16" else 0.0, HALF_STEP[dtype])
    assert not out[:, 0].any() and torch.all(lse[0] == -torch.inf) and not got[0][:, 0].any()
    for name, g in zip(("out", "lse", "dq", "dk", "dv", "dbias"), (out, lse, *got)):
        check(name, g, vals[name], tol[name])


@pytest.mark.gpu
def test_bias_strides_and_types():
    """A transposed bf16 table of more buckets than the plan uses gives its fp32 copy's result."""
    from vlm_zigzag_head_gb300 import ScorePlan, cp_attn_scored_bwd, cp_attn_scored_fwd, relative_buckets
    H, d, cu = 3, 64, [0, 200]
    q, k, v, dout = (x.to(DEV) for x in _inputs(200, H, 3, d, "bf16", 8))
    plan = ScorePlan(cu, H, rel_buckets=relative_buckets(8, 64), device=DEV)
    t = torch.randn(10, H, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    a = cp_attn_scored_fwd(q, k, v, plan, R64, rel_bias=t.t())
    b = cp_attn_scored_fwd(q, k, v, plan, R64, rel_bias=t.t().float().contiguous())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    db = cp_attn_scored_bwd(q, k, v, *a, dout, plan, R64, rel_bias=t.t())[3]
    assert db.shape == (H, 10) and not db[:, 8:].any()


@pytest.mark.gpu
@pytest.mark.parametrize("H,Hkv", [(4, 1), (3, 1), (2, 2)])
def test_bf16_gradients_are_the_rounded_fp32_ones(H, Hkv):
    """Shared groups (summed by atomics: up to the order of fp32 sums) and whole ones."""
    from vlm_zigzag_head_gb300 import CpError, ScorePlan, cp_attn_scored_bwd, cp_attn_scored_fwd
    q, k, v, dout = (x.to(DEV) for x in _inputs(333, H, Hkv, 64, "bf16", 3))
    plan = ScorePlan([0, 200, 333], H, rel_buckets=[0, 1, 2], device=DEV)
    bias = torch.randn(H, 3, device=DEV).to(torch.bfloat16)
    out, lse, lo = cp_attn_scored_fwd(q, k, v, plan, R64, rel_bias=bias, residual=True)
    a = cp_attn_scored_bwd(q, k, v, out, lse, dout, plan, R64, rel_bias=bias, out_lo=lo)
    b = cp_attn_scored_bwd(q, k, v, out, lse, dout, plan, R64, rel_bias=bias, out_lo=lo, grad_dtype=torch.bfloat16)
    for x, y in zip(a, b):
        assert x.dtype == torch.float32 and y.dtype == torch.bfloat16
        # half a step of bf16, and the sums' own variation (1e-5 of the largest)
        assert torch.all((x - y.float()).abs() <= 2.0 ** -8 * x.abs() + 1e-5 * x.abs().max())
    with pytest.raises(CpError):
        cp_attn_scored_bwd(q.float(), k.float(), v.float(), out.float(), lse, dout.float(), plan, R64,
                           grad_dtype=torch.bfloat16)


@pytest.mark.gpu
def test_plain_scores_equal_the_unmodified_attention():
    """Without cap and bias the causal result is cp_attn_fwd's, up to its summation order."""
    from vlm_zigzag_head_gb300 import ScorePlan, cp_attn_bwd, cp_attn_fwd, cp_attn_scored_bwd, cp_attn_scored_fwd
    cu, N, H, d = [0, 64 + 512], 64, 2, 128
    q, k, v, dout = (x.to(DEV) for x in _inputs(cu[-1], H, 1, d, "bf16", 4))
    plan = ScorePlan(cu, H, prefix_len=N, device=DEV)
    a = cp_attn_scored_fwd(q, k, v, plan, R128, residual=True)
    b = cp_attn_fwd(q, k, v, cu, 2, N, R128, residual=True)
    assert (a[0].float() - b[0].float()).abs().max() < 2e-2 and (a[1] - b[1]).abs().max() < 1e-4
    ga = cp_attn_scored_bwd(q, k, v, a[0], a[1], dout, plan, R128, out_lo=a[2])
    gb = cp_attn_bwd(q, k, v, b[0], b[1], dout, cu, 2, N, R128, out_lo=b[2])
    for x, y in zip(ga, gb):
        assert (x - y).norm() <= 5e-3 * y.norm()


@pytest.mark.gpu
def test_autograd_norm_rope_into_scored_attention():
    """The two operators as a model runs them: projection output -> norm and rotation -> attention with
    a cap and a learned bias -> gradients of the projection output, the norm weights and the bias."""
    from vlm_zigzag_head_gb300 import ScorePlan, relative_buckets
    from vlm_zigzag_head_gb300.autograd import cp_attention_scored, qk_norm_rope
    H, Hkv, d, cu, N = 4, 2, 64, [0, 150, 210], 33
    T, g = cu[-1], torch.Generator().manual_seed(12)
    x = torch.randn(T, H + 2 * Hkv, d, generator=g).to(torch.bfloat16)
    qw, kw = 1 + 0.2 * torch.randn(d, generator=g), 1 + 0.2 * torch.randn(d, generator=g)
    buckets = relative_buckets(16, 64)
    bias = torch.randn(H, 16, generator=g)
    dout = torch.randn(T, H, d, generator=g).to(torch.bfloat16)
    pos = torch.cat([torch.arange(150), torch.arange(60)]).to(torch.int32)
    leaves = [t.to(DEV).requires_grad_(True) for t in (x, qw, kw, bias)]
    plan = ScorePlan(cu, H, prefix_len=N, bidirectional_prefix=True, rel_buckets=buckets, device=DEV)
    xd = leaves[0]
    qn, kn = qk_norm_rope(xd[:, :H], xd[:, H:H + Hkv], pos.to(DEV), leaves[1], leaves[2])
    out, lse = cp_attention_scored(qn, kn, xd[:, H + Hkv:], plan, softcap=15.0, rel_bias=leaves[3])
    got = torch.autograd.grad(out, leaves, dout.to(DEV))
    # the chain in 64 bits, with q and k rounded to bf16 between the operators as above
    freqs = [10000.0 ** (-2.0 * p / d) for p in range(d // 2)]
    tail = (1e-6, d, freqs, [d // 2], False)
    x64 = O._f64(x)
    q64 = O.norm_rope_fwd(x64[:, :H], pos, qw, *tail)
    k64 = O.norm_rope_fwd(x64[:, H:H + Hkv], pos, kw, *tail)
    s = O.Scores(softcap=15.0, bias=bias, buckets=buckets, prefix_lens=[N, N], bidirectional=True)
    o64, lse64, dq, dk, dv, db = O.scored_attention(q64, k64, x64[:, H + Hkv:], cu, d ** -0.5, s, dout)
    dxq, dqw = O.norm_rope_bwd(x64[:, :H], dq, pos, qw, *tail)
    dxk, dkw = O.norm_rope_bwd(x64[:, H:H + Hkv], dk, pos, kw, *tail)
    want = (np.concatenate([dxq, dxk, dv], axis=1), dqw, dkw, db)
    # five roundings to bf16 lie between x and its gradient (q or k, P, dS, dq, dx): 5 x 2^-8 in norm
    for name, a, b in zip(("out", "dx", "dqw", "dkw", "dbias"), (out, *got), (o64, *want)):
        err = np.linalg.norm(O._f64(a) - b) / np.linalg.norm(b)
        assert err <= 5 * 2.0 ** -8, (name, err)
    assert np.abs(O._f64(lse) - lse64).max() < 0.05


@pytest.mark.gpu
def test_autograd_without_gradients_and_partial_leaves():
    from vlm_zigzag_head_gb300 import ScorePlan
    from vlm_zigzag_head_gb300.autograd import cp_attention_scored
    cu, H, d = [0, 90], 2, 64
    q, k, v, dout = (x.to(DEV) for x in _inputs(90, H, 2, d, "bf16", 6))
    plan = ScorePlan(cu, H, device=DEV)
    slopes = torch.tensor([0.5, 0.25], device=DEV)
    out0, lse0 = cp_attention_scored(q, k, v, plan, slopes=slopes)
    assert not out0.requires_grad
    vl = v.clone().requires_grad_(True)
    out, lse = cp_attention_scored(q, k, vl, plan, slopes=slopes)
    assert torch.equal(out, out0) and torch.equal(lse, lse0) and not lse.requires_grad
    (dv,) = torch.autograd.grad(out, vl, dout.float().to(torch.bfloat16))
    assert dv.dtype == torch.bfloat16 and dv.shape == v.shape


@pytest.mark.gpu
def test_streams_graphs_and_shared_plans():
    """One plan under two streams at once and in two captured graphs that replay in turn."""
    from vlm_zigzag_head_gb300 import ScorePlan, cp_attn_scored_bwd, cp_attn_scored_fwd
    cu, H, d = [0, 300, 500], 4, 64
    plan = ScorePlan(cu, H, rel_buckets=[0, 1, 2, 3], device=DEV)
    bias = torch.randn(H, 4, device=DEV)
    sets = [[x.to(DEV) for x in _inputs(500, H, 2, d, "bf16", s)] for s in (1, 2)]

    def both(x):
        out, lse, lo = cp_attn_scored_fwd(*x[:3], plan, R64, softcap=5.0, rel_bias=bias, residual=True)
        return (out, lse) + cp_attn_scored_bwd(*x[:3], out, lse, x[3], plan, R64, softcap=5.0, rel_bias=bias,
                                               out_lo=lo)

    def same(a, b):     # out, lse bit by bit; the summed gradients up to the order of fp32 sums
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        for x, y in zip(a[2:], b[2:]):
            assert (x - y).norm() <= 1e-5 * y.norm()
    want = [[t.clone() for t in both(x)] for x in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        got = []
        for st, x in zip(streams, sets):
            with torch.cuda.stream(st):
                got.append(both(x))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        same(a, b)
    graphs, held = [], []
    for x in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held.append(both(x))
        graphs.append(g)
    for x in sets:
        x[0].neg_()
    for g in graphs + graphs:
        g.replay()
    torch.cuda.synchronize()
    for a, x in zip(held, sets):
        same(a, both(x))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kw", [dict(), dict(softcap=4.0), dict(slopes=True), dict(bias=True),
                                dict(softcap=4.0, bias=True)])
@pytest.mark.parametrize("d", [64, 128])
def test_nan_and_infinity_stay_in_their_sample(dtype, kw, d):
    """A sample of NaN and infinities between two others: those get the bits they get beside a finite
    one (gradients up to the order of fp32 sums; under a cap an infinity in a shared tile may select
    the other evaluation of tanh, 1e-6 apart, which can turn a rounding to bf16).  Lengths end inside
    tiles; the prefix is two-way."""
    from vlm_zigzag_head_gb300 import ScorePlan, cp_attn_scored_bwd, cp_attn_scored_fwd
    lens, H = [150, 70, 131], 4
    cu, opt = _cu(lens), {}
    plan = ScorePlan(cu, H, prefix_len=[40, 70, 5], bidirectional_prefix=True, rel_buckets=[0, 1, 2, 2, 3], device=DEV)
    if "softcap" in kw:
        opt["softcap"] = kw["softcap"]
    if "slopes" in kw:
        opt["slopes"] = torch.tensor([0.5, 0.25, 0.1, 0.01], device=DEV)
    if "bias" in kw:
        opt["rel_bias"] = torch.randn(H, 4, device=DEV, generator=torch.Generator(DEV).manual_seed(1))

    def run(x):
        out, lse, *lo = cp_attn_scored_fwd(*x[:3], plan, R64, residual=dtype == "bf16", **opt)
        return [out, lse.t()] + list(cp_attn_scored_bwd(*x[:3], out, lse, x[3], plan, R64,
                                                        out_lo=lo[0] if lo else None, **opt))[:3]
    clean = [x.to(DEV) for x in _inputs(cu[-1], H, 2, d, dtype, 6)]
    dirty = [x.clone() for x in clean]
    for i, x in enumerate(dirty):
        x[150:220] = float("nan")
        x[150 + 7 * i:220:13] = float("inf")
    for i, (a, b) in enumerate(zip(run(clean), run(dirty))):
        for rows in (slice(0, 150), slice(220, 351)):
            x, y = a[rows].float(), b[rows].float()
            assert torch.isfinite(y).all(), i
            if "softcap" in kw and i < 2:
                assert torch.all((x - y).abs() <= 2.0 ** -7 * x.abs() + 1e-5), i
            elif i < 2:
                assert torch.equal(x, y), i
            else:   # dS rounded to bf16 on the other side of a border: one step of 2^-8 in few places
                assert (x - y).norm() <= (2.0 ** -10 if "softcap" in kw else 1e-5) * x.norm(), i


@pytest.mark.gpu
def test_no_tokens_and_given_outputs():
    from vlm_zigzag_head_gb300 import CpError, ScorePlan, cp_attn_scored_bwd, cp_attn_scored_fwd
    H, d = 2, 64
    plan = ScorePlan([0, 0, 0], H, rel_buckets=[0, 1], device=DEV)
    e = [torch.zeros(0, H, d, dtype=torch.bfloat16, device=DEV) for _ in range(4)]
    bias = torch.randn(H, 2, device=DEV)
    out, lse = cp_attn_scored_fwd(*e[:3], plan, R64, rel_bias=bias)
    got = cp_attn_scored_bwd(*e[:3], out, lse, e[3], plan, R64, rel_bias=bias)
    assert out.shape == (0, H, d) and not got[3].any()
    plan = ScorePlan([0, 70], H, device=DEV)
    q, k, v, dout = (x.to(DEV) for x in _inputs(70, H, 1, d, "bf16", 2))
    out, lse = torch.empty_like(q), torch.empty(H, 70, device=DEV)
    a = cp_attn_scored_fwd(q, k, v, plan, R64, softcap=3.0, out=out, lse=lse)
    assert a[0] is out and a[1] is lse
    for bad in (dict(out=out[:60]), dict(lse=lse.double()), dict(slopes=torch.ones(3, device=DEV)),
                dict(slopes=torch.ones(H)), dict(rel_bias=torch.ones(H, 2, device=DEV)),
                dict(softcap=-1.0), dict(softcap=float("nan"))):
        with pytest.raises(CpError):
            cp_attn_scored_fwd(q, k, v, plan, R64, **bad)
    for args in ((q[:60], k[:60], v[:60]), (q.half(), k.half(), v.half()), (q, k.float(), v), (q, k, v[:, :, :32]),
                 (q.transpose(0, 1), k, v), (q[0], k, v)):
        with pytest.raises(CpError):
            cp_attn_scored_fwd(*args, plan, R64)


@pytest.mark.gpu
def test_bounds_checked_build_meets_no_index_outside_a_tensor():
    from vlm_zigzag_head_gb300 import build
    from vlm_zigzag_head_gb300._binding import bounds_checked
    build.build(checked=True)
    with bounds_checked():
        _run([300, 1, 129], [40, 0, 129], True, 4, 2, 64, "bf16", R64, 8.0, "slopes", seed=1)
        _run([260], 0, False, 2, 2, 128, "bf16", R128, 0.0, (8, 64), seed=2)


@pytest.mark.gpu
def test_waits_that_give_up_on_tiles_with_foreign_rows():
    """The same with tiles that end inside a sample (their loads land on barriers of their own), forward
    and backward; the next calls are exact again."""
    from vlm_zigzag_head_gb300 import ScorePlan, Workspace, cp_attn_scored_bwd, cp_attn_scored_fwd, cp_set_wait_limit
    from vlm_zigzag_head_gb300 import cp_workspace_status
    cu = _cu([300, 77, 500, 1])
    q, k, v, dout = (x.to(DEV) for x in _inputs(cu[-1], 4, 2, 128, "bf16", 1))
    plan = ScorePlan(cu, 4, prefix_len=1, bidirectional_prefix=True, device=DEV)
    ws = Workspace(DEV)

    def both():
        out, lse, lo = cp_attn_scored_fwd(q, k, v, plan, R128, softcap=5.0, workspace=ws, residual=True)
        a = cp_workspace_status(ws)
        g = cp_attn_scored_bwd(q, k, v, out, lse, dout, plan, R128, softcap=5.0, workspace=ws, out_lo=lo)
        return a, cp_workspace_status(ws), (out, lse) + g
    want = both()
    assert want[:2] == (0, 0)
    cp_set_wait_limit(1)
    try:
        seen = [both()[:2] for _ in range(3)]
    finally:
        cp_set_wait_limit(0)
    assert any(7 in s for s in seen) and all(x in (0, 7) for s in seen for x in s)
    got = both()
    assert got[:2] == (0, 0) and torch.equal(got[2][0], want[2][0]) and torch.equal(got[2][1], want[2][1])
    for x, y in zip(got[2][2:], want[2][2:]):
        assert (x - y).norm() <= 1e-5 * y.norm()


@pytest.mark.gpu
def test_strided_inputs_and_broadcast_bias_through_autograd():
    """q, k, v as slices of one tensor that start off the 16-byte grid, a bias row shared by all heads
    (expanded), and slopes that ask for a gradient."""
    from vlm_zigzag_head_gb300 import CpError, ScorePlan
    from vlm_zigzag_head_gb300.autograd import cp_attention_scored
    H, Hkv, d, T = 4, 2, 64, 150
    g = torch.Generator().manual_seed(4)
    x = torch.randn(T, H + 2 * Hkv, d + 3, generator=g).to(torch.bfloat16).to(DEV)[..., 1:d + 1].requires_grad_(True)
    row = torch.randn(1, 3, generator=g).to(DEV).requires_grad_(True)
    plan = ScorePlan([0, 90, T], H, rel_buckets=[0, 1, 2], device=DEV)
    dout = torch.randn(T, H, d, generator=g).to(torch.bfloat16).to(DEV)
    out, _ = cp_attention_scored(x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:], plan, rel_bias=row.expand(H, 3))
    dx, drow = torch.autograd.grad(out, (x, row), dout)
    ops = [t.detach().contiguous().requires_grad_(True) for t in (x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:])]
    full = row.detach().expand(H, 3).contiguous().requires_grad_(True)
    out2, _ = cp_attention_scored(*ops, plan, rel_bias=full)
    got = torch.autograd.grad(out2, ops + [full], dout)
    assert torch.equal(out, out2)
    for a, b in ((dx, torch.cat(got[:3], dim=1)), (drow, got[3].sum(0, keepdim=True))):
        assert (a.float() - b.float()).norm() <= 2.0 ** -8 * b.float().norm()
    with pytest.raises(CpError):
        cp_attention_scored(*ops, plan, slopes=torch.ones(H, device=DEV, requires_grad=True))


@pytest.mark.gpu
def test_fp32_bias_of_bf16_inputs_and_back():
    """The bias keeps its own dtype, in its gradient too."""
    from vlm_zigzag_head_gb300 import ScorePlan
    from vlm_zigzag_head_gb300.autograd import cp_attention_scored
    plan = ScorePlan([0, 70], 2, rel_buckets=[0, 1, 2], device=DEV)
    for dtype, bdtype in (("bf16", torch.float32), ("f32", torch.bfloat16)):
        q, k, v, dout = (x.to(DEV) for x in _inputs(70, 2, 2, 64, dtype, 2))
        bias = torch.randn(2, 3, device=DEV).to(bdtype).requires_grad_(True)
        out, _ = cp_attention_scored(q, k, v, plan, rel_bias=bias)
        (db,) = torch.autograd.grad(out, bias, dout)
        s = O.Scores(bias=bias.detach().cpu(), buckets=[0, 1, 2])
        vals, tol = reference(q, k, v, [0, 70], 64 ** -0.5, s, dout, HALF_STEP["bf16"] if dtype == "bf16" else 0.0,
                              HALF_STEP[dtype])
        assert db.dtype == bdtype
        check("dbias", db, vals["dbias"], tol["dbias"], extra=torch.finfo(bdtype).eps / 2)


@pytest.mark.gpu
def test_wait_that_gives_up_is_reported():
    """With the shortest wait limit the kernels leave early and the status says so."""
    from vlm_zigzag_head_gb300 import ScorePlan, Workspace, cp_attn_scored_fwd, cp_set_wait_limit, cp_workspace_status
    q, k, v, _ = (x.to(DEV) for x in _inputs(2048, 2, 2, 128, "bf16", 1))
    plan = ScorePlan([0, 2048], 2, device=DEV)
    ws = Workspace(DEV)
    cp_set_wait_limit(1)
    try:
        cp_attn_scored_fwd(q, k, v, plan, R128, softcap=5.0, workspace=ws)
        assert cp_workspace_status(ws) == 7
    finally:
        cp_set_wait_limit(0)
    cp_attn_scored_fwd(q, k, v, plan, R128, softcap=5.0, workspace=ws)
    assert cp_workspace_status(ws) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["slopes", "bias"])
def test_saved_tensors_that_come_back_with_other_strides(kind):
    """Offloading moves what the backward needs and keeps contiguous copies: a transposed bias too."""
    from vlm_zigzag_head_gb300 import ScorePlan
    from vlm_zigzag_head_gb300.autograd import cp_attention_scored
    H, d, T = 3, 64, 75
    plan = ScorePlan([0, 40, T], H, rel_buckets=[0, 1, 2, 2, 3], device=DEV)
    q, k, v, dout = (x.to(DEV) for x in _inputs(T, H, H, d, "f32", 7))
    leaves = [x.requires_grad_(True) for x in (q, k, v)]
    opt = dict(slopes=torch.tensor([0.5, 0.25, 0.1], device=DEV))
    if kind == "bias":
        bias = torch.randn(4, H, device=DEV, generator=torch.Generator(DEV).manual_seed(2)).t().requires_grad_(True)
        leaves.append(bias)
        opt = dict(rel_bias=bias)
    want = torch.autograd.grad(cp_attention_scored(q, k, v, plan, **opt)[0], leaves, dout)
    with torch.autograd.graph.save_on_cpu():
        out, _ = cp_attention_scored(q, k, v, plan, **opt)
    got = torch.autograd.grad(out, leaves, dout)
    # equal up to the order of the atomic sums
    assert all((a - b).norm() <= 1e-5 * b.norm() for a, b in zip(got, want))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_offsets_past_32_bits(dtype):
    """The last sample of tensors with more than 2^31 elements gets the bits that it gets alone
    (two key tiles at most add to a row of dq, and two addends have one sum)."""
    from vlm_zigzag_head_gb300 import ScorePlan, cp_attn_scored_bwd, cp_attn_scored_fwd
    H, d, n, m = 64, 64, 120, 512
    before = 2 ** 31 // (H * d)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator(DEV).manual_seed(3)
    tails = [torch.randn((n, H, d), device=DEV, generator=g).to(dt) for _ in range(4)]
    slopes = torch.linspace(0.01, 0.5, H, device=DEV)
    ends = []
    for T in (before + n, n):
        plan = ScorePlan(list(range(0, T - n + 1, m)) + [T], H, device=DEV)
        x = [torch.zeros((T, H, d), dtype=dt, device=DEV) for _ in range(4)]
        for a, b in zip(x, tails):
            a[-n:] = b
        out, lse, lo = cp_attn_scored_fwd(*x[:3], plan, R64, slopes=slopes, residual=True)
        got = cp_attn_scored_bwd(*x[:3], out, lse, x[3], plan, R64, slopes=slopes, out_lo=lo, grad_dtype=dt)
        ends.append([t[-n:].clone() for t in (out, lse.t(), *got)])
    for a, b in zip(*ends):
        assert torch.isfinite(a).all()
        if dtype == "bf16":
            assert torch.equal(a, b)
        else:   # the walk of the sample alone may be shared between blocks
            assert (a - b).norm() <= 1e-5 * b.norm()
    del x, out, lse, lo, got, plan
    torch.cuda.empty_cache()


@pytest.mark.gpu
@pytest.mark.parametrize("bias", [False, True])
def test_small_gradients_beside_a_sample_that_is_not_finite(bias):
    """f16 operands are scaled by their tensor's largest finite value: gradients of 1e-7 beside a
    sample of NaN and infinities equal those beside a finite one."""
    from vlm_zigzag_head_gb300 import ScorePlan, cp_attn_scored_bwd, cp_attn_scored_fwd
    cu, H, d = [0, 140, 210, 300], 2, 64
    plan = ScorePlan(cu, H, rel_buckets=[0, 1, 2], device=DEV)
    opt = dict(rel_bias=torch.randn(H, 3, device=DEV, generator=torch.Generator(DEV).manual_seed(1))) if bias else {}
    clean = [x.to(DEV) for x in _inputs(cu[-1], H, 1, d, "bf16", 8)]
    for x, f in zip(clean, (1e-2, 1e-2, 1e-6, 1e-7)):
        x *= f
    dirty = [x.clone() for x in clean]
    for x in clean:
        x[140:210] = 0
    for i, x in enumerate(dirty):
        x[140:210] = float("nan")
        x[140 + i:210:9] = float("-inf")
    ends = []
    for x in (clean, dirty):
        out, lse, lo = cp_attn_scored_fwd(*x[:3], plan, 1.0, residual=True, **opt)
        got = cp_attn_scored_bwd(*x[:3], out, lse, x[3], plan, 1.0, out_lo=lo, **opt)
        ends.append([torch.cat([t[:140], t[210:]]).float() for t in (out, lse.t(), *got[:3])])
    for a, b in zip(*ends):
        assert a.norm() > 0 and (a - b).norm() <= 1e-5 * a.norm()


CUT = [   # one or two heads: runs of more than three tiles are cut into parts
    ([1500], 0, False, 1, 1, 64, R64, 0.0, "slopes"),
    ([1111, 130], 0, False, 2, 1, 128, R128, 20.0, None),
    ([1300, 77], [300, 77], True, 2, 2, 64, R64, 0.0, (32, 1000)),
    ([1200], 700, True, 1, 1, 128, R128, 5.0, "slopes"),
    ([1025, 0, 1], [1, 0, 1], True, 3, 1, 64, 1.0, 4.0, (8, 32)),      # f16 operands
    ([1400], 0, False, 1, 1, 128, R128, 0.0, (8, 16)),
]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,prefix,both,H,Hkv,d,scale,cap,kind", CUT)
def test_cut_runs_match_oracle(lens, prefix, both, H, Hkv, d, scale, cap, kind):
    gain = 1.0 if scale < 0.5 else d ** -0.5
    _run(lens, prefix, both, H, Hkv, d, "bf16", scale, cap, kind, gain, seed=len(lens))


@pytest.mark.gpu
def test_cut_runs_whose_parts_see_nothing():
    """A bias that hides near or far keys leaves whole parts, and some rows, without a key."""
    from vlm_zigzag_head_gb300 import ScorePlan, cp_attn_scored_bwd, cp_attn_scored_fwd
    H, d, cu = 3, 64, [0, 1290]
    buckets = [0] * 200 + [1] * 200 + [2]
    bias = torch.zeros(H, 3)
    bias[0, 1:] = float("-inf")     # the last parts alone
    bias[1, :2] = float("-inf")     # the first parts; rows below 400 see nothing
    bias[2, :] = float("-inf")
    q, k, v, dout = _inputs(cu[-1], H, 1, d, "bf16", 5)
    plan = ScorePlan(cu, H, rel_buckets=buckets, device=DEV)
    dv = [x.to(DEV) for x in (q, k, v, dout)]
    out, lse, lo = cp_attn_scored_fwd(*dv[:3], plan, R64, rel_bias=bias.to(DEV), residual=True)
    got = cp_attn_scored_bwd(*dv[:3], out, lse, dv[3], plan, R64, rel_bias=bias.to(DEV), out_lo=lo)
    s = O.Scores(bias=bias.clamp(min=-1e38), buckets=buckets)
    vals, tol = reference(q, k, v, cu, R64, s, dout, HALF_STEP["bf16"], HALF_STEP["bf16"])
    assert not out[:400, 1].any() and not out[:, 2].any()
    assert torch.all(lse[1, :400] == -torch.inf) and torch.all(lse[2] == -torch.inf)
    for name, g in zip(("out", "lse", "dq", "dk", "dv", "dbias"), (out, lse, *got)):
        check(name, g, vals[name], tol[name])


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["cap", "slopes", "bias"])
def test_cut_runs_keep_samples_apart(kind):
    """NaN in the samples around a cut one, a captured call, and bf16 gradients."""
    from vlm_zigzag_head_gb300 import ScorePlan, cp_attn_scored_bwd, cp_attn_scored_fwd
    H, d, cu = 2, 64, [0, 70, 1270, 1500]
    plan = ScorePlan(cu, H, rel_buckets=[0, 1, 2], device=DEV)
    opt = {"cap": dict(softcap=6.0), "slopes": dict(slopes=torch.tensor([0.1, 0.02], device=DEV)),
           "bias": dict(rel_bias=torch.randn(H, 3, device=DEV, generator=torch.Generator(DEV).manual_seed(1)))}[kind]
    x = [t.to(DEV) for t in _inputs(cu[-1], H, 1, d, "bf16", 8)]

    def run():
        out, lse, lo = cp_attn_scored_fwd(*x[:3], plan, R64, residual=True, **opt)
        return (out, lse.t()) + cp_attn_scored_bwd(*x[:3], out, lse, x[3], plan, R64, out_lo=lo,
                                                   grad_dtype=torch.bfloat16, **opt)[:3]
    want = [t.clone() for t in run()]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = run()
    for t in x:
        t[:70] = float("nan")
        t[1270:] = float("inf")
    g.replay()
    torch.cuda.synchronize()
    for i, (a, b) in enumerate(zip(want, held)):
        a, b = a[70:1270].float(), b[70:1270].float()
        assert torch.isfinite(b).all(), i
        # an infinity in a shared tile may select the other evaluation of tanh; sums in another order turn
        # a rounding to bf16 in few places
        assert (a - b).norm() <= 2.0 ** -10 * a.norm(), i


@pytest.mark.gpu
def test_bounds_checked_build_meets_no_index_outside_a_tensor_in_cut_runs():
    from vlm_zigzag_head_gb300 import build
    from vlm_zigzag_head_gb300._binding import bounds_checked
    build.build(checked=True)
    with bounds_checked():
        _run([1300, 1, 129], [40, 0, 129], True, 2, 1, 64, "bf16", R64, 8.0, "slopes", seed=1)
        _run([1060], 0, False, 1, 1, 128, "bf16", R128, 0.0, (8, 64), seed=2)


@pytest.mark.gpu
@pytest.mark.parametrize("scale,cap", [(1e-8, 1e-3), (1e-8, 1e4), (0.2, 1e4), (0.2, 1e-3), (20.0, 1e4), (1e-3, 1e-3)])
@pytest.mark.parametrize("kind", [None, "slopes", (8, 32)])
def test_ends_of_the_cap_and_scale_ranges(scale, cap, kind):
    """Coefficients of the cap's polynomial that would leave the range of normal numbers."""
    _run([150, 33], 0, False, 2, 1, 64, "bf16", scale, cap, kind, 1.0 if scale < 1 else 0.125, seed=3)


@pytest.mark.gpu
@pytest.mark.parametrize("lens,H,Hkv", [([130], 6, 2), ([200, 40], 5, 1), ([1100], 6, 1), ([90], 12, 2)])
def test_groups_that_are_no_power_of_two(lens, H, Hkv):
    _run(lens, 0, False, H, Hkv, 64, "bf16", R64, 20.0, "slopes", seed=H)


@pytest.mark.gpu
@pytest.mark.parametrize("longest", [1024, 1025])
def test_both_operand_types_of_the_backward(longest):
    """The longest sample decides between f16 and bf16 dS: both within the bounds, with a short one beside."""
    _run([longest, 60], [9, 5], True, 4, 2, 64, "bf16", R64, 0.0, (8, 32), seed=2)
