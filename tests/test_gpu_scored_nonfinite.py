"""Query rows of NaN or infinities, and scores that overflow: out, lse and dq of the row are NaN however its
keys are shared out, as the formula gives; a row that sees no key stays apart from them."""
import os
import subprocess
import sys

import pytest
import torch

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _inputs(T, H, Hkv, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn((T, h, d), generator=g).to(DT[dtype]).to(DEV) for h in (H, Hkv, Hkv, H)]


SHAPES = [   # lens, prefix, H, Hkv, dtype
    ([1500], 0, 1, 1, "bf16"),          # keys cut into parts that are joined
    ([1300, 77], 300, 2, 1, "bf16"),
    ([300, 129], 20, 8, 2, "bf16"),     # whole runs
    ([700], 0, 2, 1, "f32"),            # walks shared by blocks, merged
    ([300, 65], 64, 2, 2, "f32"),
    ([64] * 400, 0, 8, 8, "f32"),       # one block a walk
]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,prefix,H,Hkv,dtype", SHAPES)
@pytest.mark.parametrize("kind,what", [(k, w) for k in ("plain", "cap", "slopes", "bias")
                                       for w in ("nan", "overflow") if (k, w) != ("cap", "overflow")])
def test_rows_that_are_not_finite(lens, prefix, H, Hkv, dtype, kind, what):
    from vlm_zigzag_head_gb300 import ScorePlan, cp_attn_scored_bwd, cp_attn_scored_fwd
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    d = 64
    pre = [min(prefix, n) for n in lens]
    plan = ScorePlan(cu, H, prefix_len=pre, bidirectional_prefix=True, rel_buckets=[0, 1, 2], device=DEV)
    opt = {"plain": {}, "cap": dict(softcap=6.0), "slopes": dict(slopes=torch.linspace(0.01, 0.2, H, device=DEV)),
           "bias": dict(rel_bias=torch.randn(H, 3, device=DEV, generator=torch.Generator(DEV).manual_seed(1)))}[kind]
    x = _inputs(cu[-1], H, Hkv, d, dtype, 5)

    def run():
        out, lse, *lo = cp_attn_scored_fwd(*x[:3], plan, 0.125, residual=True, **opt)
        got = cp_attn_scored_bwd(*x[:3], out, lse, x[3], plan, 0.125, out_lo=lo[0] if lo else None, **opt)
        return out, lse, got[0], got[1], got[2]
    want = [t.clone() for t in run()]
    bad = sorted({3, min(250, cu[1] - 1), cu[1] - 2})     # rows of head 0 in the first sample
    for i in bad:
        if what == "nan":
            x[0][i, 0] = float("nan")
        else:   # the product with key 1 (or 2) is far above the largest fp32 number
            x[0][i, 0] = 1e38 * x[1][1 + i % 2, 0].sign()
    got = run()
    assert torch.isnan(got[0][bad, 0]).all() and torch.isnan(got[1][0, bad]).all()
    assert torch.isnan(got[2][bad, 0]).all()
    # every other row of out and lse keeps its bits (under a cap a NaN in the tile changes none)
    for a, b in ((want[0], got[0]), (want[1].t(), got[1].t())):
        a, b = a.clone(), b.clone()
        a[bad, 0] = b[bad, 0] = 0
        assert torch.equal(a, b)
    # keys that a bad row sees have no finite gradient (other products may overflow to minus infinity, which
    # hides the key); the next sample's are as before
    assert torch.isnan(got[3][slice(0, 4) if what == "nan" else slice(1, 3), 0]).all()
    for a, b in zip(want[2:], got[2:]):
        a, b = a[cu[1]:], b[cu[1]:]
        assert torch.isfinite(b).all() and (a - b).norm() <= 1e-5 * a.norm()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 66])
def test_merge_keeps_nan_beside_parts_that_saw_nothing(d):
    """Row 0: NaN and -inf; row 1: NaN and a finite lse; row 2: -inf alone; row 3: finite alone."""
    from vlm_zigzag_head_gb300 import cp_lse_merge
    nan, inf = float("nan"), float("inf")
    lse = torch.tensor([[nan, 1.0, -inf, 0.5], [-inf, nan, -inf, -inf], [-inf, 2.0, -inf, 0.25]], device=DEV)[:, None]
    part = torch.ones(3, 4, 1, d, device=DEV)
    part[0, 0] = part[1, 1] = nan
    out, got = cp_lse_merge(part, lse.contiguous())
    assert torch.isnan(out[:2]).all() and torch.isnan(got[0, :2]).all()
    assert not out[2].any() and got[0, 2] == -inf
    assert (out[3] - 1).abs().max() < 1e-6 and torch.isfinite(got[0, 3])


def _unmodified():
    from vlm_zigzag_head_gb300 import cp_attn_fwd
    q, k, v, _ = _inputs(64 + 512, 2, 2, 128, "bf16", 2)
    want = cp_attn_fwd(q, k, v, [0, 576], 2, 64, 128 ** -0.5)
    bad = [10, 64, 300, 575]
    q[bad, 1] = float("nan")
    out, lse = cp_attn_fwd(q, k, v, [0, 576], 2, 64, 128 ** -0.5)
    assert torch.isnan(out[bad, 1]).all() and torch.isnan(lse[1, bad]).all()
    out[bad, 1], lse[1, bad] = want[0][bad, 1], want[1][1, bad]
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.gpu
def test_unmodified_attention_reports_nan_too():
    """The kernels are shared: the rank-wise forward writes the same lse, in one launch and in one per ring
    step (chosen once per process, so in a child)."""
    _unmodified()
    code = "import sys; sys.path[:0] = %r; import test_gpu_scored_nonfinite as t; t._unmodified()" % [
        os.path.dirname(os.path.dirname(os.path.abspath(__file__))), os.path.dirname(os.path.abspath(__file__))]
    r = subprocess.run([sys.executable, "-c", code], env=dict(os.environ, CPATTN_FWD_PER_STEP="1"),
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
