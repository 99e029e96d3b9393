"""The activations of fp32 calls keep fp32's digits, in their tails too.

Tolerances, derived from the arithmetic; u = 2^-24, and every product of these calls has a single term
that is a value times 1, so all of them are exact.  silu: the exponential is off by at most two units in
the last place (4 u of its value), the sum with 1 by 5 u then, its inverse by 6 u: that is the sigmoid s;
a = g s by 7 u.  a' = s + a (1 - s) adds 6 u s, 8 u |a| and u |a'|.  gelu_tanh: the sigmoid's argument
z = k g (1 + 0.044715 g^2) carries five roundings, constants among them: 5 u |z| of s more (1 - s is off by
as much of s), and a' = s + a (1 - s) z' another 5 u of z' = k (1 + 0.134145 g^2).  Terms of second
order: 10 % more."""
import numpy as np
import pytest
import torch

from gpu_util import to64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24


def _reference(g, act):
    """a, a', and the bounds of their errors, in 64 bits."""
    if act == "silu":
        z, slope, carried = g, np.ones_like(g), np.zeros_like(g)
    else:
        k = 2 * np.sqrt(2 / np.pi)
        z, slope = k * (g + 0.044715 * g ** 3), k * (1 + 0.134145 * g * g)
        carried = 5 * np.abs(z)
    e = np.exp(-np.abs(z))
    s, rest = np.where(z < 0, e, 1) / (1 + e), np.where(z < 0, 1, e) / (1 + e)
    a = g * s
    da = s + a * rest * slope
    ea = 1.1 * U * (7 + carried * rest) * np.abs(a)
    eda = 1.1 * U * ((6 + carried * rest) * s + (8 + 2 * carried + 5 * (act != "silu")) * np.abs(a) * slope +
                     np.abs(da))
    return a, da, ea, eda


@pytest.mark.parametrize("act,low", [("silu", -60.0), ("gelu_tanh", -5.0)])
@pytest.mark.parametrize("T", [1, 2, 4, 8, 24, 25, 64, 65, 300, 4000])   # every kernel of fp32 rows
def test_activations_of_single_terms(T, act, low):
    import vlm_zigzag_head_gb300 as cp
    g = torch.linspace(low, 0.5 * -low, T, device=DEV) if T > 1 else torch.full((1,), 0.8 * low, device=DEV)
    x = torch.zeros(T, 8, device=DEV)
    x[:, 0], x[:, 1] = g, 1.0
    wg, wu, wd = (torch.zeros(8, 8, device=DEV) for _ in range(3))
    wg[0, 0] = wu[0, 1] = wd[0, 0] = 1.0
    dy = torch.ones(T, 8, device=DEV)
    y, gate, up = cp.cp_gated_ffn_fwd(x, wg, wu, wd, act, keep=True)
    dx = cp.cp_gated_ffn_bwd(x, wg, wu, wd, gate, up, dy, act)[0]
    a, da, ea, eda = _reference(to64(g), act)
    for name, got, want, tol in (("y", y, a, ea), ("dx", dx, da, eda)):
        err = np.abs(to64(got)[:, 0] - want)
        assert np.all(err <= tol), (name, float((err / tol).max()), float(to64(g)[np.argmax(err / tol)]))
    err = np.abs(to64(dx)[:, 1] - a)
    assert np.all(err <= ea), float((err / ea).max())
