"""The fp64 oracles of the norm with rotation and of scored attention, pinned on the CPU: their
gradients equal central differences of their forwards, and simple cases equal closed forms."""
import numpy as np
import pytest

from oracle import scored as O


def _freqs(rot, theta=10000.0):
    return [theta ** (-2.0 * p / rot) for p in range(rot // 2)]


def _differences(f, x, g, count, seed, step=1e-5):
    """Central differences of sum(f(x) * g) at some elements of x."""
    rng = np.random.default_rng(seed)
    out = []
    for flat in rng.choice(x.size, size=min(count, x.size), replace=False):
        e = np.zeros(x.size)
        e[flat] = step
        e = e.reshape(x.shape)
        out.append((flat, float(((f(x + e) - f(x - e)) * g).sum() / (2 * step))))
    return out


@pytest.mark.parametrize("rot,sections,inter", [(16, [8], False), (16, [8], True), (8, [1, 3], False),
                                                (0, [0], False)])
def test_norm_rope_gradient_is_the_difference_quotient(rot, sections, inter):
    rng = np.random.default_rng(1)
    T, H, d = 3, 2, 16
    x, dy, w = rng.normal(size=(T, H, d)), rng.normal(size=(T, H, d)), rng.normal(size=d)
    pos = rng.integers(0, 1000, size=(len(sections), T))
    args = (1e-3, rot, _freqs(rot) if rot else [], sections, inter)
    dx, dw = O.norm_rope_bwd(x, dy, pos, w, *args)
    for flat, want in _differences(lambda z: O.norm_rope_fwd(z, pos, w, *args), x, dy, 40, 2):
        assert abs(dx.reshape(-1)[flat] - want) < 1e-7
    for flat, want in _differences(lambda z: O.norm_rope_fwd(x, pos, z, *args), w, dy, 16, 3):
        assert abs(dw[flat] - want) < 1e-7


def test_norm_rope_keeps_the_norm_and_turns_by_the_distance():
    """With unit weights the rotation keeps the RMS, and products depend on the distance alone."""
    rng = np.random.default_rng(4)
    d = 16
    q, k = rng.normal(size=(1, 1, d)), rng.normal(size=(1, 1, d))
    dots = []
    for a, b in ((5, 2), (100005, 100002)):
        y = O.norm_rope_fwd(q, [[a]], None, 0.0, d, _freqs(d), [d // 2], False)
        z = O.norm_rope_fwd(k, [[b]], None, 0.0, d, _freqs(d), [d // 2], False)
        assert abs((y * y).mean() - 1) < 1e-12
        dots.append(float((y * z).sum()))
    assert abs(dots[0] - dots[1]) < 1e-9


SCORES = [
    dict(softcap=2.0),
    dict(slopes=np.array([0.5, 0.01])),
    dict(bias=np.array([[0.1, -0.3, 0.2], [1.0, 0.0, -1.0]]), buckets=[0, 1, 1, 2]),
    dict(softcap=1.5, slopes=np.array([0.3, 0.1]), prefix_lens=(3, 2), bidirectional=True),
    dict(softcap=1.5, bias=np.array([[0.1, -0.3, 0.2], [1.0, 0.0, -1.0]]), buckets=[0, 1, 1, 2],
         prefix_lens=(3, 0), bidirectional=True),
]


@pytest.mark.parametrize("spec", SCORES)
def test_scored_gradients_are_difference_quotients(spec):
    rng = np.random.default_rng(7)
    cu, H, Hkv, d = [0, 6, 11], 2, 1, 4
    q, dout = rng.normal(size=(11, H, d)), rng.normal(size=(11, H, d))
    k, v = rng.normal(size=(11, Hkv, d)), rng.normal(size=(11, Hkv, d))
    s = O.Scores(**spec)
    _, _, dq, dk, dv, dbias = O.scored_attention(q, k, v, cu, 0.7, s, dout)
    for name, x, grad in (("q", q, dq), ("k", k, dk), ("v", v, dv)):
        def f(z, name=name):
            a = dict(q=q, k=k, v=v)
            a[name] = z
            return O.scored_attention(a["q"], a["k"], a["v"], cu, 0.7, s)[0]
        for flat, want in _differences(f, x, dout, 30, 8):
            assert abs(grad.reshape(-1)[flat] - want) < 1e-7, name
    if s.bias is not None:
        def f(z):
            return O.scored_attention(q, k, v, cu, 0.7, s._replace(bias=z))[0]
        for flat, want in _differences(f, s.bias, dout, 6, 9):
            assert abs(dbias.reshape(-1)[flat] - want) < 1e-7


def test_scored_masks():
    rng = np.random.default_rng(3)
    q, k, v = (rng.normal(size=(5, 1, 4)) for _ in range(3))
    # a prefix that sees itself both ways: row 0 of a prefix of 3 averages rows 0..2
    out, lse = O.scored_attention(q, k, v, [0, 5], 0.0,
                                  O.Scores(prefix_lens=(3,), bidirectional=True))
    assert np.allclose(out[0, 0], v[:3, 0].mean(0)) and np.allclose(lse[0, 0], np.log(3))
    assert np.allclose(out[3, 0], v[:4, 0].mean(0))
    # a bias that hides every distance leaves rows empty; one that hides distance 0 the first row
    hid = O.Scores(bias=np.array([[-np.inf, -3.4e38]]), buckets=[0, 1])
    out, lse, dq, dk, dv, db = O.scored_attention(q, k, v, [0, 5], 1.0, hid, v)
    assert not out.any() and np.all(lse == -np.inf) and not dq.any() and not dv.any()
    one = O.Scores(bias=np.array([[-3.4e38, 0.0]]), buckets=[0, 1])
    out, lse = O.scored_attention(q, k, v, [0, 5], 1.0, one)
    assert not out[0].any() and lse[0, 0] == -np.inf and np.allclose(out[1], v[0])
