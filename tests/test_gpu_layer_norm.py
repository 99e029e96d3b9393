"""Layer norm and its gradient against the fp64 oracle.

Tolerances, derived from the arithmetic.  u = 2^-24 (half a step of fp32).  A row's sum is added
by at most 64 elements a thread, 5 shuffles and 32 warps: 101 u times the sum of magnitudes, so the
mean is off by at most 101 u mean|x|, and every x - mean by that plus u |x - mean|.  The sum of
squares is off by 101 u relative from its own sums and by the mean's error twice, the root by half
of it plus 2 u: with m = mean|x| r (how far the row lies from zero, in deviations), n is off by at
most (101 m + |n| (52 + 101 m + 4)) u.  The weight adds 2 u of the value.  Backward: the sums of g
and g n add 101 u of mean|g| and mean|g n| and the error of n; dx is off by at most
r (u (105 + 202 (1 + m)) (|g| + mean|g| + (1 + |n|) mean|g n| + |n| mean|g|)).  A weight gradient
adds at most T + 64 terms: (T + 64) u times the sum of magnitudes, and the error of n.  A result in
bf16 adds half a step of bf16, 2^-8 of the value."""
import numpy as np
import pytest
import torch

from gpu_util import to64
from oracle import layer as O

DEV = "cuda:0"
U = 2.0 ** -24
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _inputs(T, D, dtype, layout, seed, offset=0.3):
    g = torch.Generator().manual_seed(seed)
    pad = {"plain": 0, "sliced": 64, "odd": 3}[layout]
    x = torch.randn((T, D + pad), generator=g) * (1 + torch.rand((T, 1), generator=g)) + offset
    x[:, ::max(1, D // 4)] *= 8
    dy = torch.randn((T, D + pad), generator=g)
    x, dy = x.to(dtype).to(DEV), dy.to(dtype).to(DEV)
    skip = 1 if layout == "odd" else pad
    w, b = 1 + 0.3 * torch.randn(D, generator=g), 0.3 * torch.randn(D, generator=g)
    return x[:, skip:skip + D], dy[:, skip:skip + D], w.to(DEV), b.to(DEV)


def _tolerances(x, w, b, eps):
    x = to64(x)
    y, mean, rstd = O.layer_norm_fwd(x, w, b, eps)
    n = O.layer_norm_fwd(x, None, None, eps)[0]
    m = np.abs(x).mean(-1, keepdims=True) * rstd[:, None]
    err_n = U * (101 * m + np.abs(n) * (56 + 101 * m))
    w64 = np.ones(x.shape[1]) if w is None else to64(w)
    err_y = err_n * np.abs(w64) + 2 * U * (np.abs(n * w64) + np.abs(y))
    return n, rstd[:, None], m, err_n, err_y


def _check_fwd(y, x, w, b, eps, dtype):
    want = O.layer_norm_fwd(x, w, b, eps)[0]
    tol = _tolerances(x, w, b, eps)[4] + HALF_STEP[dtype] * np.abs(want)
    err = np.abs(to64(y) - want)
    assert np.all(err <= tol), float((err / np.maximum(tol, 1e-300)).max())


def _check_bwd(dx, dw, db, x, dy, w, eps, dtype):
    n, r, m, err_n, _ = _tolerances(x, w, None, eps)
    wdx, wdw, wdb = O.layer_norm_bwd(x, dy, w, eps)
    d = to64(dy)
    g = d if w is None else d * to64(w)
    if dx is not None:
        ag, agn = np.abs(g).mean(-1, keepdims=True), np.abs(g * n).mean(-1, keepdims=True)
        tol = r * U * (105 + 202 * (1 + m)) * (np.abs(g) + ag + (1 + np.abs(n)) * agn + np.abs(n) * ag)
        tol = tol + HALF_STEP[dtype] * np.abs(wdx)
        err = np.abs(to64(dx) - wdx)
        assert np.all(err <= tol), float((err / np.maximum(tol, 1e-300)).max())
    T = x.shape[0]
    if dw is not None:
        tol = (T + 64) * U * np.abs(d * n).sum(0) + (np.abs(d) * err_n).sum(0)
        err = np.abs(to64(dw) - wdw)
        assert np.all(err <= tol), float((err / np.maximum(tol, 1e-300)).max())
    if db is not None:
        assert np.all(np.abs(to64(db) - wdb) <= (T + 64) * U * np.abs(d).sum(0))


# every width class of the kernels in both types, vector and element loads
CASES = [(1, 4096, "bf16", "plain"), (3, 16, "bf16", "plain"), (9, 1, "f32", "plain"), (37, 7, "bf16", "odd"),
         (5, 1000, "f32", "plain"), (19, 1000, "bf16", "sliced"), (700, 64, "bf16", "plain"),
         (33, 333, "f32", "odd"), (65, 2048, "bf16", "sliced"), (11, 2049, "bf16", "plain"),
         (330, 4096, "bf16", "plain"), (7, 4096, "f32", "odd"), (13, 8192, "bf16", "plain"),
         (5, 8191, "f32", "plain"), (3, 16384, "bf16", "sliced"), (310, 16384, "f32", "plain"),
         (4, 16381, "f32", "odd"), (6, 12000, "bf16", "odd"), (2500, 512, "f32", "plain"),
         (17, 5120, "f32", "sliced"), (21, 511, "bf16", "plain"), (9, 4100, "bf16", "plain")]


@pytest.mark.gpu
@pytest.mark.parametrize("T,D,dtype,layout", CASES)
def test_matches_oracle(T, D, dtype, layout):
    import vlm_zigzag_head_gb300 as cp
    dt = DT[dtype]
    x, dy, w, b = _inputs(T, D, dt, layout, T + D)
    y, mean, rstd = cp.cp_layer_norm_fwd(x, w, b)
    assert y.dtype == dt and y.is_contiguous() and y.shape == x.shape
    _check_fwd(y, x, w, b, 1e-5, dt)
    _check_fwd(cp.cp_layer_norm_fwd(x)[0], x, None, None, 1e-5, dt)
    dx, dw, db = cp.cp_layer_norm_bwd(x, dy, mean, rstd, w, bias_grad=True)
    _check_bwd(dx, dw, db, x, dy, w, 1e-5, dt)
    again = cp.cp_layer_norm_bwd(x, dy, mean, rstd, w, bias_grad=True)
    assert all(torch.equal(a, c) for a, c in zip((dx, dw, db), again))
    dx, dw, db = cp.cp_layer_norm_bwd(x, dy, mean, rstd)
    assert dw is None and db is None
    _check_bwd(dx, None, None, x, dy, None, 1e-5, dt)


@pytest.mark.gpu
def test_parts_that_are_wanted():
    import vlm_zigzag_head_gb300 as cp
    x, dy, w, b = _inputs(40, 256, torch.bfloat16, "plain", 1)
    _, mean, rstd = cp.cp_layer_norm_fwd(x, None, b)
    full = cp.cp_layer_norm_bwd(x, dy, mean, rstd, w, bias_grad=True)
    for inp in (False, True):
        for wg in (False, True):
            for bg in (False, True):
                got = cp.cp_layer_norm_bwd(x, dy, mean, rstd, w, input_grad=inp, weight_grad=wg, bias_grad=bg)
                for have, want, on in zip(got, full, (inp, wg, bg)):
                    assert (have is None) if not on else torch.equal(have, want)


@pytest.mark.gpu
def test_bf16_weights_leading_dimensions_and_no_rows():
    import vlm_zigzag_head_gb300 as cp
    x, dy, w, b = _inputs(24, 320, torch.bfloat16, "plain", 2)
    w, b = w.to(torch.bfloat16), b.to(torch.bfloat16)
    y, mean, rstd = cp.cp_layer_norm_fwd(x.view(2, 3, 4, 320), w, b)
    assert y.shape == (2, 3, 4, 320) and mean.shape == (2, 3, 4)
    _check_fwd(y.view(24, 320), x, w, b, 1e-5, torch.bfloat16)
    dx, dw, db = cp.cp_layer_norm_bwd(x.view(6, 4, 320), dy.view(6, 4, 320), mean, rstd, w, bias_grad=True)
    _check_bwd(dx.view(24, 320), dw, db, x, dy, w, 1e-5, torch.bfloat16)
    y1, m1, r1 = cp.cp_layer_norm_fwd(x[0], w, b)          # a single row without a token dimension
    assert y1.shape == (320,) and torch.equal(y1, y.view(24, 320)[0])
    # transposed storage is copied
    xt = x.t().contiguous().t()
    assert torch.equal(cp.cp_layer_norm_fwd(xt, w, b)[0], y.view(24, 320))
    e, em, er = cp.cp_layer_norm_fwd(x[:0], w, b)
    assert e.shape == (0, 320)
    dx, dw, db = cp.cp_layer_norm_bwd(x[:0], dy[:0], em, er, w, bias_grad=True)
    assert dx.shape == (0, 320) and not dw.any() and not db.any()


@pytest.mark.gpu
def test_far_means_equal_rows_and_nan_stay_in_their_row():
    """A row whose mean is 1000 times its spread keeps its digits (no difference of squares); a
    constant row is zero; a NaN or an infinity reaches its own row alone."""
    import vlm_zigzag_head_gb300 as cp
    x, dy, w, b = _inputs(12, 1024, torch.float32, "plain", 3, offset=1000.0)
    y, mean, rstd = cp.cp_layer_norm_fwd(x, w, b)
    _check_fwd(y, x, w, b, 1e-5, torch.float32)
    x, dy, w, b = _inputs(12, 1024, torch.bfloat16, "plain", 4)
    clean, cm, cr = cp.cp_layer_norm_fwd(x, w, b)
    cdx = cp.cp_layer_norm_bwd(x, dy, cm, cr, w)[0]
    bad = x.clone()
    bad[2, 5], bad[4, 1000], bad[7] = float("nan"), float("inf"), 2.0
    y, mean, rstd = cp.cp_layer_norm_fwd(bad, w, b)
    dx = cp.cp_layer_norm_bwd(bad, dy, mean, rstd, w)[0]
    same = [i for i in range(12) if i not in (2, 4, 7)]
    assert torch.equal(y[same], clean[same]) and torch.equal(dx[same], cdx[same])
    assert y[2].isnan().all() and y[4].isnan().any() and torch.equal(y[7], b.to(torch.bfloat16))


@pytest.mark.gpu
def test_autograd_streams_and_devices_of_use():
    """Gradients through autograd equal the formula's and differences; a call on another stream
    and a captured, replayed pair of calls give the same bits."""
    import vlm_zigzag_head_gb300 as cp
    from vlm_zigzag_head_gb300.autograd import layer_norm
    x, dy, w, b = _inputs(30, 200, torch.float32, "sliced", 5)
    leaves = [t.detach().clone().requires_grad_(True) for t in (x, w, b)]
    y = layer_norm(*leaves)
    dx, dw, db = torch.autograd.grad(y, leaves, dy)
    _check_bwd(dx, dw, db, x, dy, w, 1e-5, torch.float32)
    # a central difference along a direction, in 64 bits by the oracle at x +- h v
    v = np.random.default_rng(0).standard_normal(x.shape)
    h = 1e-5
    plus, minus = (O.layer_norm_fwd(to64(x) + s * h * v, w, b, 1e-5)[0] for s in (1, -1))
    slope = ((plus - minus) / (2 * h) * to64(dy)).sum()
    scale = np.abs(to64(dx) * v).sum()
    assert abs((to64(dx) * v).sum() - slope) <= 1e-5 * scale
    # an expanded gradient (a sum's) and a frozen weight
    gx, = torch.autograd.grad(layer_norm(leaves[0], w).sum(), leaves[0])
    assert torch.equal(gx, cp.cp_layer_norm_bwd(x, torch.ones_like(dy), *cp.cp_layer_norm_fwd(x, w)[1:], w)[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ys, ms, rs = cp.cp_layer_norm_fwd(x, w, b)
        gs = cp.cp_layer_norm_bwd(x, dy, ms, rs, w, bias_grad=True)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(ys, y) and all(torch.equal(a, c) for a, c in zip(gs, (dx, dw, db)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        yg, mg, rg = cp.cp_layer_norm_fwd(x, w, b)
        gg = cp.cp_layer_norm_bwd(x, dy, mg, rg, w, bias_grad=True)
    for _ in range(2):
        for t in (yg, *gg):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(yg, y) and all(torch.equal(a, c) for a, c in zip(gg, (dx, dw, db)))


@pytest.mark.gpu
def test_rows_beyond_32_bit_offsets():
    """A view whose last rows start past 2^31 elements."""
    import vlm_zigzag_head_gb300 as cp
    big = torch.zeros((3, (1 << 30) + 512), dtype=torch.bfloat16, device=DEV)
    x = big[:, :256]
    x.copy_(torch.randn(3, 256))
    y, mean, rstd = cp.cp_layer_norm_fwd(x)
    want, wm, wr = cp.cp_layer_norm_fwd(x.contiguous())
    assert torch.equal(y, want)
    assert torch.equal(cp.cp_layer_norm_bwd(x, x, mean, rstd)[0],
                       cp.cp_layer_norm_bwd(x.contiguous(), x.contiguous(), wm, wr)[0])
