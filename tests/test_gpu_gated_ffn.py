"""Gated feed-forward block and its gradient against the fp64 oracle.

Tolerances, derived from the arithmetic.  b = 2^-8 is half a step of bf16, u = 2^-24 of fp32; r is
b for bf16 calls and u for fp32 ones.  A product of length K adds its terms in fp32, each addition
off by at most a step (the tensor core may cut off): 2 (K + 8) u times the sum of magnitudes.  The
activation is off by 2^-20 of its value (exponential 2 u, its argument's rounding times up to 32,
division 2 u).  Slopes: |a'| <= 1.13, |a''| <= 1.  With e_z the error of z, forward:
    e_h <= 1.13 e_g |u| + |a| (e_u + 2^-20 |u|) + r |h|,  e_y = e_h |Wd| + sum error + r |y|;
backward, from g and u kept to 24 bits (e_g + k |g|, e_u + k |u|; k = 2^-15 in bf16, 0 in fp32):
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
    k = 0.0 if r == U else 2.0 ** -15
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
         (8, 40, 24, 56, "bf16", "gelu"), (20, 8, 16, 24, "bf16", "silu"), (9, 2048, 6144, 2048, "bf16", "silu"), (31, 264, 1000, 1032, "bf16", "silu"),
         (33, 136, 520, 72, "bf16", "gelu_tanh"), (64, 512, 1040, 512, "bf16", "gelu"),
         (65, 512, 1040, 512, "bf16", "gelu"), (100, 2048, 520, 1000, "bf16", "silu"),
         (127, 264, 4104, 264, "bf16", "gelu_tanh"),
         (2500, 1536, 768, 1280, "bf16", "gelu_tanh"), (5000, 1024, 1280, 1024, "bf16", "silu"),
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


# dx, the two weights' and the down weight's gradients are one launch: dx first with its k shared; all
# whole in two rounds; dx last, behind fp32 gradients of the weights; a few tiles each; one long product
ONE_LAUNCH = [(700, 320, 1664, 320, "silu"), (2000, 512, 1360, 520, "gelu"), (6000, 520, 64, 264, "silu"),
              (30, 512, 1360, 512, "gelu_tanh"), (9000, 1032, 136, 40, "silu"), (400, 64, 8000, 72, "silu"),
              (150, 1920, 3968, 24, "silu")]


@pytest.mark.gpu
@pytest.mark.parametrize("T,D,F,D_out,act", ONE_LAUNCH)
def test_gradients_of_one_launch(T, D, F, D_out, act):
    import vlm_zigzag_head_gb300 as cp
    dt = torch.bfloat16
    x, wg, wu, wd, dy = _inputs(T, D, F, D_out, dt, T + D + F)
    y, gate, up = cp.cp_gated_ffn_fwd(x, wg, wu, wd, act, keep=True)
    ws = cp.Workspace()
    for grad_dtype in (torch.float32, dt):
        full = cp.cp_gated_ffn_bwd(x, wg, wu, wd, gate, up, dy, act, grad_dtype=grad_dtype, workspace=ws)
        assert cp.cp_workspace_status(ws) == 0
        _check((y, *full), x, wg, wu, wd, dy, act, dt, grad_dtype)
        for wanted in ((True, False, False, True), (True, True, False, False), (False, True, True, True)):
            some = cp.cp_gated_ffn_bwd(x, wg, wu, wd, gate, up, dy, act, grad_dtype=grad_dtype,
                                       wanted=list(wanted), workspace=ws)
            assert cp.cp_workspace_status(ws) == 0
            _check((y, *some), x, wg, wu, wd, dy, act, dt, grad_dtype)


def _call(seed=1, T=70, D=72, F=136, D_out=40, dtype=torch.bfloat16):
    import vlm_zigzag_head_gb300 as cp
    x, wg, wu, wd, dy = _inputs(T, D, F, D_out, dtype, seed)
    y, gate, up = cp.cp_gated_ffn_fwd(x, wg, wu, wd, keep=True)
    return cp, x, wg, wu, wd, dy, y, gate, up


@pytest.mark.gpu
@pytest.mark.parametrize("T,D,F", [(70, 72, 136), (700, 2048, 2304)])   # the second: shared last tiles
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_parts_that_are_wanted(T, D, F, dtype):
    cp, x, wg, wu, wd, dy, y, gate, up = _call(2, T, D, F, 104, dtype)
    ws = cp.Workspace()
    full = cp.cp_gated_ffn_bwd(x, wg, wu, wd, gate, up, dy, grad_dtype=dtype)
    for bits in range(16):
        wanted = [bool(bits >> i & 1) for i in range(4)]
        got = cp.cp_gated_ffn_bwd(x, wg, wu, wd, gate, up, dy, grad_dtype=dtype, wanted=wanted, workspace=ws)
        for have, want, on in zip(got, full, wanted):
            assert (have is None) == (not on)
            # one weight alone shares its k otherwise than both: other roundings of the sums
            assert not on or rel_l2(have, want) <= 2 * (F32_REL if dtype == torch.float32 else 2.0 ** -8)
    if ws.buf is not None:
        assert cp.cp_workspace_status(ws) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strided_rows_halves_of_one_weight_and_no_rows(dtype):
    """Rows out of wider ones and one [2 F][D] weight give the bits of contiguous copies; nothing beside
    the outputs is written."""
    import vlm_zigzag_head_gb300 as cp
    T, D, F, Do = 150, 72, 136, 40
    x, wg, wu, wd, dy = _inputs(T, D, F, Do, dtype, 3)
    both = torch.cat([wg, wu])
    xs = torch.full((T, D + 24), float("nan"), dtype=dtype, device=DEV)[:, 8:8 + D]
    dys = torch.full((T, Do + 16), float("nan"), dtype=dtype, device=DEV)[:, 16:]
    wds = torch.full((Do, F + 8), float("nan"), dtype=dtype, device=DEV)[:, :F]
    for to, frm in ((xs, x), (dys, dy), (wds, wd)):
        to.copy_(frm)
    y, g, u = cp.cp_gated_ffn_fwd(x, wg, wu, wd, keep=True)
    grads = cp.cp_gated_ffn_bwd(x, wg, wu, wd, g, u, dy)
    ys, gs, us = cp.cp_gated_ffn_fwd(xs, both[:F], both[F:], wds, keep=True)
    assert torch.equal(y, ys)
    for a, b in zip(grads, cp.cp_gated_ffn_bwd(xs, both[:F], both[F:], wds, gs, us, dys)):
        assert torch.equal(a, b)
    # leading dimensions, and none
    y3, g3, u3 = cp.cp_gated_ffn_fwd(x.view(5, 30, D), wg, wu, wd, keep=True)
    assert y3.shape == (5, 30, Do) and torch.equal(y3.view(T, Do), y)
    dx3 = cp.cp_gated_ffn_bwd(x.view(5, 30, D), wg, wu, wd, g3, u3, dy.view(5, 30, Do))[0]
    assert dx3.shape == (5, 30, D) and torch.equal(dx3.view(T, D), grads[0])
    assert cp.cp_gated_ffn_fwd(x[7], wg, wu, wd).shape == (Do,)
    y0, g0, u0 = cp.cp_gated_ffn_fwd(x[:0], wg, wu, wd, keep=True)
    assert y0.shape == (0, Do)
    zero = cp.cp_gated_ffn_bwd(x[:0], wg, wu, wd, g0, u0, dy[:0])
    assert zero[0].shape == (0, D) and not any(z.any() for z in zero[1:])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,act", [(torch.bfloat16, "silu"), (torch.float32, "gelu"), (torch.float32, "gelu_tanh")])
def test_autograd_against_formula_and_differences(dtype, act):
    from vlm_zigzag_head_gb300.autograd import gated_ffn
    T, D, F, Do = 60, 64, 128, 48
    x, wg, wu, wd, dy = _inputs(T, D, F, Do, dtype, 4)
    leaves = [t.clone().requires_grad_(True) for t in (x, wg, wu, wd)]
    y = gated_ffn(*leaves, activation=act)
    grads = torch.autograd.grad(y, leaves, dy)
    _check((y, *grads), x, wg, wu, wd, dy, act, dtype, dtype)
    # a central difference along a random direction of all inputs, in 64 bits by the oracle
    rng, h = np.random.default_rng(0), 1e-5
    args = [to64(t) for t in (x, wg, wu, wd)]
    dirs = [rng.standard_normal(a.shape) * np.abs(a).mean() for a in args]
    plus, minus = (O.gated_ffn(*(a + s * h * v for a, v in zip(args, dirs)), act) for s in (1, -1))
    slope = ((plus - minus) / (2 * h) * to64(dy)).sum()
    got = sum((to64(g) * v).sum() for g, v in zip(grads, dirs))
    size = sum(np.linalg.norm(to64(g)) * np.linalg.norm(v) for g, v in zip(grads, dirs))
    assert abs(got - slope) <= (BF16_REL if dtype == torch.bfloat16 else 2 * F32_REL) * size
    # frozen weights, rows off the 16-byte grid, an expanded gradient
    odd = torch.zeros((T, D + 1), dtype=dtype, device=DEV)[:, 1:]
    odd.copy_(x)
    odd.requires_grad_(True)
    dx, = torch.autograd.grad(gated_ffn(odd, wg, wu, wd, activation=act), odd, dy[:1].expand(T, Do))
    dx2, = torch.autograd.grad(gated_ffn(leaves[0], wg, wu, wd, activation=act), leaves[0],
                               dy[:1].expand(T, Do).contiguous())
    assert torch.equal(dx, dx2)


@pytest.mark.gpu
@pytest.mark.parametrize("T,D,F", [(60, 64, 128), (1, 256, 512), (400, 1024, 768)])
def test_streams_and_graphs(T, D, F):
    """Calls on several streams at once, and captured ones replayed, give the same bits."""
    cp, x, wg, wu, wd, dy, y, gate, up = _call(5, T, D, F, 128)
    grads = cp.cp_gated_ffn_bwd(x, wg, wu, wd, gate, up, dy)
    sides, got = [torch.cuda.Stream() for _ in range(3)], []
    torch.cuda.synchronize()
    for s in sides:
        with torch.cuda.stream(s):
            r = cp.cp_gated_ffn_fwd(x, wg, wu, wd, keep=True)
            got.append((r, cp.cp_gated_ffn_bwd(x, wg, wu, wd, r[1], r[2], dy)))
    torch.cuda.synchronize()
    for r, g in got:
        assert torch.equal(r[0], y) and all(torch.equal(a, b) for a, b in zip(g, grads))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        yg, gg, ug = cp.cp_gated_ffn_fwd(x, wg, wu, wd, keep=True)
        out = cp.cp_gated_ffn_bwd(x, wg, wu, wd, gg, ug, dy)
    for _ in range(2):
        for t in (yg, *out):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(yg, y) and all(torch.equal(a, b) for a, b in zip(out, grads))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 7, 300])
def test_nonfinite_rows_stay_rows(T):
    """A NaN in one row of x reaches that row of y and dx alone, and every weight gradient."""
    cp, x, wg, wu, wd, dy, y, gate, up = _call(6, T)
    clean = cp.cp_gated_ffn_bwd(x, wg, wu, wd, gate, up, dy)
    row = T // 2
    bad = x.clone()
    bad[row, 3] = float("nan")
    yb, gb, ub = cp.cp_gated_ffn_fwd(bad, wg, wu, wd, keep=True)
    db = cp.cp_gated_ffn_bwd(bad, wg, wu, wd, gb, ub, dy)
    keep = torch.arange(T, device=DEV) != row
    assert yb[row].isnan().all() and torch.equal(yb[keep], y[keep])
    assert db[0][row].isnan().all() and torch.equal(db[0][keep], clean[0][keep])
    assert all(d.isnan().any() for d in db[1:])


@pytest.mark.gpu
def test_large_and_tiny_values():
    """Projections far from 1 keep their digits: 24 bits at any exponent."""
    import vlm_zigzag_head_gb300 as cp
    for size in (1e-18, 1e-6, 1e6, 1e12):
        x, wg, wu, wd, dy = _inputs(40, 64, 128, 64, torch.bfloat16, 7)
        wu = (wu.float() * size).to(torch.bfloat16)
        y, g, u = cp.cp_gated_ffn_fwd(x, wg, wu, wd, keep=True)
        grads = cp.cp_gated_ffn_bwd(x, wg, wu, wd, g, u, dy)
        _check((y, *grads), x, wg, wu, wd, dy, "silu", torch.bfloat16, torch.float32)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_gates_far_out(act, dtype):
    """Where the activation is 0 or the identity: gates of both signs up to 1e30 give y = u or 0, and
    gradients that are finite and exact to their roundings."""
    import vlm_zigzag_head_gb300 as cp
    D = F = Do = 8
    for T in (4, 20, 150):
        x = torch.zeros(T, D, device=DEV)
        size = torch.logspace(2, 30, T, device=DEV)
        x[:, 0] = torch.where(torch.arange(T, device=DEV) % 2 == 0, size, -size)   # the gates
        x[:, 1] = 1.0
        wg, wu, wd = (torch.zeros(s, device=DEV) for s in ((F, D), (F, D), (Do, F)))
        wg[0, 0], wu[0, 1], wd[3, 0] = 1.0, 2.0, 1.0
        x, wg, wu, wd = (t.to(dtype) for t in (x, wg, wu, wd))
        dy = torch.ones(T, Do, dtype=dtype, device=DEV)
        y, g, u = cp.cp_gated_ffn_fwd(x, wg, wu, wd, act, keep=True)
        dx = cp.cp_gated_ffn_bwd(x, wg, wu, wd, g, u, dy, act)[0]
        gate = to64(x)[:, 0]
        step = 2 * 2.0 ** (-8 if dtype == torch.bfloat16 else -24)     # h and the result rounded
        assert np.all(np.abs(to64(y)[:, 3] - 2 * np.maximum(gate, 0)) <= step * np.abs(2 * gate) * (gate > 0))
        assert np.all(np.abs(to64(dx)[:, 0] - 2 * (gate > 0)) <= 2 * step)
        assert np.all(np.abs(to64(dx)[:, 1] - 2 * np.maximum(gate, 0)) <= step * np.abs(2 * gate) * (gate > 0))


@pytest.mark.gpu
def test_waits_that_run_out_are_reported():
    """A bounded wait cut to one polling round gives up; the status says so and the next call is exact."""
    cp, x, wg, wu, wd, dy, y, gate, up = _call(8, 600, 512, 1024, 512)
    ws, seen = cp.Workspace(), []
    cp.cp_set_wait_limit(1)
    try:
        for _ in range(3):
            cp.cp_gated_ffn_fwd(x, wg, wu, wd, workspace=ws)
            try:
                seen.append(cp.cp_workspace_status(ws))
            except cp.CpError as e:
                seen.append(e.status)
    finally:
        cp.cp_set_wait_limit(0)
    assert all(s in (0, 7) for s in seen) and 7 in seen, seen
    assert torch.equal(cp.cp_gated_ffn_fwd(x, wg, wu, wd, workspace=ws), y)
    assert cp.cp_workspace_status(ws) == 0


# ---- fp32 of more than 64 rows: factors as three bf16 values, six products of them

SPLIT = [(65, 72, 136, 40, "silu"), (517, 512, 1360, 512, "gelu"), (700, 2048, 264, 520, "silu"),
         (2500, 136, 72, 264, "gelu_tanh"), (300, 8, 8, 8, "silu"), (128, 1024, 2816, 1032, "silu"),
         (1100, 520, 1032, 264, "silu")]


@pytest.mark.gpu
@pytest.mark.parametrize("T,D,F,D_out,act", SPLIT)
def test_fp32_of_many_rows(T, D, F, D_out, act):
    import vlm_zigzag_head_gb300 as cp
    x, wg, wu, wd, dy = _inputs(T, D, F, D_out, torch.float32, T + D + F)
    ws = cp.Workspace()
    y, gate, up = cp.cp_gated_ffn_fwd(x, wg, wu, wd, act, keep=True, workspace=ws)
    assert cp.cp_workspace_status(ws) == 0
    assert torch.equal(cp.cp_gated_ffn_fwd(x, wg, wu, wd, act), y)
    full = cp.cp_gated_ffn_bwd(x, wg, wu, wd, gate, up, dy, act, workspace=ws)
    assert cp.cp_workspace_status(ws) == 0
    _check((y, *full), x, wg, wu, wd, dy, act, torch.float32, torch.float32)
    again = cp.cp_gated_ffn_bwd(x, wg, wu, wd, gate, up, dy, act)
    assert all(torch.equal(a, b) for a, b in zip(full, again))
    for wanted in ((True, False, False, True), (False, True, False, False), (False, False, True, True)):
        some = cp.cp_gated_ffn_bwd(x, wg, wu, wd, gate, up, dy, act, wanted=list(wanted), workspace=ws)
        assert cp.cp_workspace_status(ws) == 0
        _check((y, *some), x, wg, wu, wd, dy, act, torch.float32, torch.float32)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [72, 200, 520])
@pytest.mark.parametrize("scale", [2.0 ** -60, 1.0, 2.0 ** 60])
def test_fp32_keeps_all_digits(n, scale):
    """Products with a single term that is a value times a power of two give the value's 24 bits:
    no part of it is lost.  silu(128) = 128 and silu'(128) = 1 in fp32 (e^-128 < 2^-126)."""
    import vlm_zigzag_head_gb300 as cp
    g = torch.Generator().manual_seed(n)
    eye = torch.eye(n, device=DEV)
    values, dy = ((torch.randn(n, n, generator=g) * scale).to(DEV) for _ in range(2))
    x, wg, wu = 128 * eye, eye, eye / 16384          # g = 128 on the diagonal, u = 1 / 128, h = 1
    y, gate, up = cp.cp_gated_ffn_fwd(x, wg, wu, values, keep=True)
    assert torch.equal(y, values.t())
    dwd = cp.cp_gated_ffn_bwd(x, wg, wu, values, gate, up, dy, wanted=[False, False, False, True])[3]
    assert torch.equal(dwd, dy.t())
    # the down weight an identity: dh = dy, of which the diagonal goes on: dg = dy / 128, du = 128 dy
    dx, dwg, dwu, _ = cp.cp_gated_ffn_bwd(x, wg, wu, eye, gate, up, dy)
    diag = torch.diag(torch.diag(dy))
    assert torch.equal(dx, diag / 64) and torch.equal(dwg, diag) and torch.equal(dwu, diag * 16384)
    # rows of 24 bits: u = x / 128 where the gates are 128
    up_w, rows = torch.zeros(n, n + 8, device=DEV), torch.zeros(n, n + 8, device=DEV)
    gate_w = torch.zeros(n, n + 8, device=DEV)
    gate_w[:, 0] = 128.0
    rows[:, 0], rows[:, 8:], up_w[:, 8:] = 1.0, values, eye / 128
    assert torch.equal(cp.cp_gated_ffn_fwd(rows, gate_w, up_w, eye), values)


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_fp32_nonfinite_rows_stay_rows(bad):
    cp, x, wg, wu, wd, dy, y, gate, up = _call(6, 300, dtype=torch.float32)
    clean = cp.cp_gated_ffn_bwd(x, wg, wu, wd, gate, up, dy)
    worse = x.clone()
    worse[150, 3] = bad
    yb, gb, ub = cp.cp_gated_ffn_fwd(worse, wg, wu, wd, keep=True)
    db = cp.cp_gated_ffn_bwd(worse, wg, wu, wd, gb, ub, dy)
    keep = torch.arange(300, device=DEV) != 150
    assert not yb[150].isfinite().any() and torch.equal(yb[keep], y[keep])
    assert not db[0][150].isfinite().any() and torch.equal(db[0][keep], clean[0][keep])
    assert all(not d.isfinite().all() for d in db[1:])


@pytest.mark.gpu
def test_fp32_streams_graphs_and_strides():
    cp, x, wg, wu, wd, dy, y, gate, up = _call(5, 400, 264, 768, 128, torch.float32)
    grads = cp.cp_gated_ffn_bwd(x, wg, wu, wd, gate, up, dy)
    sides, got = [torch.cuda.Stream() for _ in range(3)], []
    torch.cuda.synchronize()
    for s in sides:
        with torch.cuda.stream(s):
            r = cp.cp_gated_ffn_fwd(x, wg, wu, wd, keep=True)
            got.append((r, cp.cp_gated_ffn_bwd(x, wg, wu, wd, r[1], r[2], dy)))
    torch.cuda.synchronize()
    for r, g in got:
        assert torch.equal(r[0], y) and all(torch.equal(a, b) for a, b in zip(g, grads))
    both = torch.cat([wg, wu])                                      # halves of one weight
    wide = torch.full((400, 264 + 4), float("nan"), device=DEV)     # rows apart
    wide[:, :264] = x
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        yg, gg, ug = cp.cp_gated_ffn_fwd(wide[:, :264], both[:768], both[768:], wd, keep=True)
        out = cp.cp_gated_ffn_bwd(wide[:, :264], both[:768], both[768:], wd, gg, ug, dy)
    for _ in range(2):
        for t in (yg, *out):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(yg, y) and all(torch.equal(a, b) for a, b in zip(out, grads))


@pytest.mark.gpu
def test_fp32_waits_that_run_out_are_reported():
    cp, x, wg, wu, wd, dy, y, gate, up = _call(8, 600, 512, 1024, 512, torch.float32)
    ws, seen = cp.Workspace(), []
    cp.cp_set_wait_limit(1)
    try:
        for _ in range(3):
            cp.cp_gated_ffn_fwd(x, wg, wu, wd, workspace=ws)
            try:
                seen.append(cp.cp_workspace_status(ws))
            except cp.CpError as e:
                seen.append(e.status)
    finally:
        cp.cp_set_wait_limit(0)
    assert all(s in (0, 7) for s in seen) and 7 in seen, seen
    assert torch.equal(cp.cp_gated_ffn_fwd(x, wg, wu, wd, workspace=ws), y)
    assert cp.cp_workspace_status(ws) == 0


FEW = [(1, 8, 8, 8, "silu"), (1, 2048, 6144, 2048, "silu"), (2, 120, 136, 40, "gelu"), (3, 264, 1000, 72, "gelu_tanh"),
       (4, 1032, 264, 2048, "silu"), (5, 512, 1360, 512, "gelu"), (8, 136, 4104, 8, "silu"), (9, 40, 24, 56, "silu"),
       (16, 512, 72, 1032, "gelu_tanh"), (23, 264, 520, 264, "silu"), (24, 1000, 2048, 128, "gelu"),
       (25, 264, 520, 264, "silu"), (33, 136, 264, 72, "silu"), (64, 264, 520, 136, "gelu")]


@pytest.mark.gpu
@pytest.mark.parametrize("T,D,F,D_out,act", FEW)
def test_fp32_of_few_rows(T, D, F, D_out, act):
    import vlm_zigzag_head_gb300 as cp
    x, wg, wu, wd, dy = _inputs(T, D, F, D_out, torch.float32, T + D + F)
    ws = cp.Workspace()
    y, gate, up = cp.cp_gated_ffn_fwd(x, wg, wu, wd, act, keep=True, workspace=ws)
    assert cp.cp_workspace_status(ws) == 0
    assert torch.equal(cp.cp_gated_ffn_fwd(x, wg, wu, wd, act), y)
    grads = cp.cp_gated_ffn_bwd(x, wg, wu, wd, gate, up, dy, act, workspace=ws)
    _check((y, *grads), x, wg, wu, wd, dy, act, torch.float32, torch.float32)
    # halves of one weight, rows apart, and NaN behind them
    both, wide = torch.cat([wg, wu]), torch.full((T, D + 8), float("nan"), device=DEV)
    wide[:, :D] = x
    assert torch.equal(cp.cp_gated_ffn_fwd(wide[:, :D], both[:F], both[F:], wd, act), y)
    # a NaN in one row stays there
    bad, row = x.clone(), T // 2
    bad[row, D - 1] = float("nan")
    yb, keep = cp.cp_gated_ffn_fwd(bad, wg, wu, wd, act), torch.arange(T, device=DEV) != T // 2
    assert yb[row].isnan().all() and torch.equal(yb[keep], y[keep])


@pytest.mark.gpu
def test_fp32_single_tokens_replayed():
    """One token a step into a captured graph whose input changes, as a decoding loop has it."""
    cp, x, wg, wu, wd, dy, *_ = _call(9, 6, 512, 1360, 512, torch.float32)
    want = [cp.cp_gated_ffn_fwd(x[i:i + 1], wg, wu, wd) for i in range(6)]
    step = x[:1].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = cp.cp_gated_ffn_fwd(cp.cp_gated_ffn_fwd(step, wg, wu, wd), wg, wu, wd)
    for i in range(6):
        step.copy_(x[i:i + 1])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, cp.cp_gated_ffn_fwd(want[i], wg, wu, wd))
