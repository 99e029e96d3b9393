"""Gated feed-forward block and its gradient against the fp64 oracle.

Tolerances, derived from the arithmetic.  b = 2^-8 is half a step of bf16, u = 2^-24 of fp32; r is
b for bf16 calls and u for fp32 ones.  A product of length K adds its terms in fp32, each addition
off by at most a step (the tensor core may cut off): 2 (K + 8) u times the sum of magnitudes.  The
activation is off by 2^-20 of its value (exponential 2 u, its argument's rounding times up to 32,
division 2 u).  Slopes: |a'| <= 1.13, |a''| <= 1.  With e_z the error of z, forward:
    e_h <= 1.13 e_g |u| + |a| (e_u + 2^-20 |u|) + r |h|,  e_y = e_h |Wd| + sum error + r |y|;
backward, from g and u kept to 24 bits (e_g + k |g|, e_u + k |u|; k = 2^-17 in bf16, 0 in fp32):
    e_dg <= |u a'| e_dh + |dh a'| e_u + |dh u| (e_g + 2^-20) + r |dg|,
    e_du <= |a| e_dh + |dh| (1.13 e_g + 2^-20 |a|) + r |du|,
and the last products pass these on as y does.  Terms of second order: 10 % more.  These bounds
add magnitudes; roundings of random sign stay far below, so the relative L2 error is also held to
the method's 5e-3 (bf16) and 1e-5 (fp32)."""
import numpy as np
import pytest
import torch

from gpu_util import BF16_REL, F32_REL, rel_l2, to64
from oracle import layer as O

DEV = "cuda:0"
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def _inputs(T, D, F, D_out, dtype, seed):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g)
    x, wg, wu = normal(T, D), normal(F, D) * D ** -0.5, normal(F, D) * D ** -0.5
    wd, dy = normal(D_out, F) * F ** -0.5, normal(T, D_out)
    return [t.to(dtype).to(DEV) for t in (x, wg, wu, wd, dy)]


def _bounds(x, wg, wu, wd, dy, act, r):
    """Error bounds of y, dx, dwg, dwu, dwd before the last rounding."""
    ax, awg, awu, awd, ady = (np.abs(t) for t in (x, wg, wu, wd, dy))
    (T, D), F, Do = x.shape, wg.shape[0], wd.shape[0]

    def summed(K):
        return 2 * (K + 8) * U
    g, u = x @ wg.T, x @ wu.T
    a, da = O.activation(g, act)
    h = a * u
    eg, eu = summed(D) * (ax @ awg.T), summed(D) * (ax @ awu.T)
    eh = 1.13 * eg * np.abs(u) + np.abs(a) * (eu + 2 ** -20 * np.abs(u)) + r * np.abs(h)
    ey = eh @ awd.T + summed(F) * (np.abs(h) @ awd.T)
    k = 0.0 if r == U else 2.0 ** -17
    eg, eu = eg + k * np.abs(g), eu + k * np.abs(u)
    dh = dy @ wd
    edh = summed(Do) * (ady @ awd)
    dg, du = dh * u * da, dh * a
    edg = np.abs(u * da) * edh + np.abs(dh * da) * eu + np.abs(dh * u) * (eg + 2 ** -20) + r * np.abs(dg)
    edu = np.abs(a) * edh + np.abs(dh) * (1.13 * eg + 2 ** -20 * np.abs(a)) + r * np.abs(du)
    eh = 1.13 * eg * np.abs(u) + np.abs(a) * (eu + 2 ** -20 * np.abs(u)) + r * np.abs(h)
    adg, adu = np.abs(dg), np.abs(du)
    edx = edg @ awg + edu @ awu + summed(2 * F) * (adg @ awg + adu @ awu)
    edwg, edwu = (e.T @ ax + summed(T) * (m.T @ ax) for e, m in ((edg, adg), (edu, adu)))
    edwd = ady.T @ eh + summed(T) * (ady.T @ np.abs(h))
    return [1.1 * e for e in (ey, edx, edwg, edwu, edwd)]


def _check(got, x, wg, wu, wd, dy, act, dtype, grad_dtype):
    args = [to64(t) for t in (x, wg, wu, wd, dy)]
    want = O.gated_ffn(*args[:4], act, args[4])
    bounds = _bounds(*args, act, ROUND[dtype])
    for i, (name, have, w, e) in enumerate(zip(("y", "dx", "dw_gate", "dw_up", "dw_down"), got, want, bounds)):
        if have is None:
            continue
        last = dtype if i < 2 else grad_dtype
        assert have.dtype == last and have.is_contiguous() and have.shape == w.shape, name
        err, tol = np.abs(to64(have) - w), e + ROUND[last] * np.abs(w)
        assert np.all(err <= tol), (name, float((err / np.maximum(tol, 1e-300)).max()))
        assert rel_l2(have, w) <= (F32_REL if dtype == torch.float32 else BF16_REL), (name, rel_l2(have, w))


# tokens, width, hidden, output width; the tiles are 128 x 256 (gate and up: 128 x 128) by 64
CASES = [(1, 64, 128, 64, "bf16", "silu"), (128, 64, 128, 256, "bf16", "silu"), (2, 8, 8, 8, "bf16", "gelu"),
         (129, 72, 136, 40, "bf16", "gelu_tanh"), (300, 256, 512, 256, "bf16", "gelu"),
         (257, 520, 1032, 264, "bf16", "silu"), (37, 1024, 2816, 1024, "bf16", "gelu_tanh"),
         (3, 2048, 512, 1000, "bf16", "silu"), (16, 264, 4104, 264, "bf16", "gelu"),
         (1000, 512, 1360, 512, "bf16", "silu"), (3000, 64, 2048, 64, "bf16", "silu"),
         (2500, 1536, 768, 1280, "bf16", "gelu_tanh"),
         (1, 32, 64, 32, "f32", "silu"), (5, 8, 16, 24, "f32", "gelu"), (129, 136, 264, 72, "f32", "gelu_tanh"),
         (300, 256, 512, 256, "f32", "silu"), (17, 512, 1360, 512, "f32", "gelu"),
         (1030, 96, 200, 104, "f32", "silu")]


@pytest.mark.gpu
@pytest.mark.parametrize("T,D,F,D_out,dtype,act", CASES)
def test_matches_oracle(T, D, F, D_out, dtype, act):
    import vlm_zigzag_head_gb300 as cp
    dt = DT[dtype]
    x, wg, wu, wd, dy = _inputs(T, D, F, D_out, dt, T + D + F)
    ws = cp.Workspace()
    y, gate, up = cp.cp_gated_ffn_fwd(x, wg, wu, wd, act, keep=True, workspace=ws)
    assert cp.cp_workspace_status(ws) == 0
    assert torch.equal(cp.cp_gated_ffn_fwd(x, wg, wu, wd, act), y)
    for grad_dtype in {torch.float32, dt}:
        grads = cp.cp_gated_ffn_bwd(x, wg, wu, wd, gate, up, dy, act, grad_dtype=grad_dtype, workspace=ws)
        assert cp.cp_workspace_status(ws) == 0
        _check((y, *grads), x, wg, wu, wd, dy, act, dt, grad_dtype)
        again = cp.cp_gated_ffn_bwd(x, wg, wu, wd, gate, up, dy, act, grad_dtype=grad_dtype)
        assert all(torch.equal(a, b) for a, b in zip(grads, again))
