"""The learned bias's gradient where the probabilities of whole buckets are tiny: long rows, and buckets that
the bias itself holds down."""
import numpy as np
import pytest
import torch

from oracle import scored as O
from scored_util import check, reference

DEV = "cuda:0"
F16 = 2.0 ** -11     # half a step


@pytest.mark.gpu
@pytest.mark.parametrize("cap", [0.0, 20.0])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("down", [-6.0, -12.0])
def test_bias_gradient_of_buckets_with_tiny_probabilities(d, cap, down):
    """2048 tokens; probabilities of the held-down buckets are near 2^-17 and 2^-26.  v falls with the
    position, so that the terms of a bucket share a sign and the sum shows each one's relative error.
    The bound counts P as f16 (half a step 2^-11, here and in the forward); below 2^-28 P may lose bits
    (2^-39 each), and in the forward probabilities end at steps of 2^-24 of the row's largest."""
    from vlm_zigzag_head_gb300 import ScorePlan, cp_attn_scored_bwd, cp_attn_scored_fwd
    H, T, scale = 2, 2048, d ** -0.5
    g = torch.Generator().manual_seed(d)
    q, k = torch.randn((T, H, d), generator=g), torch.randn((T, 1, d), generator=g)
    v = 0.5 * (torch.arange(T) < 1024).float()[:, None, None] + 0.01 * torch.randn((T, 1, d), generator=g)
    dout = 0.25 + 0.01 * torch.randn((T, H, d), generator=g)
    q, k, v, dout = (x.to(torch.bfloat16) for x in (q, k, v, dout))
    buckets = [0] * 256 + [1] * 256 + [2]      # the middle one near the diagonal, the last one far
    bias = torch.tensor([[0.0, down, down], [0.25, down, down - 1]])
    plan = ScorePlan([0, T], H, rel_buckets=buckets, device=DEV)
    x = [t.to(DEV) for t in (q, k, v, dout)]
    opt = dict(softcap=cap, rel_bias=bias.to(DEV))
    out, lse, lo = cp_attn_scored_fwd(*x[:3], plan, scale, residual=True, **opt)
    dbias = cp_attn_scored_bwd(*x[:3], out, lse, x[3], plan, scale, out_lo=lo, **opt)[3]
    s = O.Scores(softcap=cap, bias=bias, buckets=buckets)
    vals, tol = reference(q, k, v, [0, T], scale, s, dout, F16, 2.0 ** -8)
    q64, k64, v64, do64 = (O._f64(t) for t in (q, k, v, dout))
    floor = np.zeros_like(vals["dbias"])
    for h in range(H):
        sc, _, seen, dist = O._sample_scores(q64[:, h], k64[:, 0], scale, s, h, 0)
        p, _ = O._softmax(sc, seen)
        dp = do64[:, h] @ v64[:, 0].T
        D = (p * dp).sum(1, keepdims=True)
        # D's own error from probabilities that end at 2^-25 of the largest
        eD = 2.0 ** -25 * (np.abs(do64[:, h]) @ np.cumsum(np.abs(v64[:, 0]), 0).T).diagonal()[:, None]
        part = seen * (2.0 ** -39 * np.abs(dp - D)) + p * eD
        np.add.at(floor[h], np.asarray(buckets)[np.minimum(np.abs(dist), 512)].ravel(), part.ravel())
    check("dbias", dbias, vals["dbias"], tol["dbias"] + floor)
    # of the held-down buckets the bound is one on precision, 2^-7 of the value at most
    assert np.all((tol["dbias"] + floor)[:, 1:] <= 2.0 ** -7 * np.abs(vals["dbias"][:, 1:]))
