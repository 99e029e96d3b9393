"""Reference values and error bounds of attention with modified scores.

Every bound is a worst case derived from the roundings, element by element, with u = 2^-24 and r the
half step of the 16-bit operands (2^-8 for bf16 P and dS; 0 on the fp32 path):

* a score is off by at most delta = (d + 16) u scale sum|q k| (fp32 sums of exact products), plus
  4e-6 of the value and of the bias (tanh, log2 units, distance times slope);
* a probability by e = 2 max delta + 2^-20 of its value (its row's normaliser errs as much; exp2);
* out by (r + e) sum p|v|, plus half a step of the output type;
* D = dout . out by eD = sum |dout| (r + e + 2^-16) sum p|v|: out is kept to 16 bits by its remainder;
* with f16 operands (softmax scale above 1/4, or short samples) dS is kept as an f16 multiple of 2^es, which ends at steps
  of 2^(es - 24): half a step, `ds_floor`, on every visible pair;
* dS = p (dP - D) w by (r + 2 e + 4e-6) |dS| + p (eD + d u sum|dout v|) + 4e-6 |p (dP - D)|;
* products of these with k, q and dout sum the bounds, and n u of the magnitudes for n summed terms.
"""
import numpy as np

from oracle import scored as O

U = 2.0 ** -24


def f16_ds_floor(v, dout):
    """es = 1 + log2 d + E_v + E_dout - 15, with E the exponents of the largest magnitudes."""
    es = 1 + np.log2(v.shape[-1]) + sum(np.frexp(np.abs(O._f64(x)).max())[1] for x in (v, dout)) - 15
    return 2.0 ** (es - 25)


def reference(q, k, v, cu, scale, s, dout, r_op, r_out, ds_floor=0.0):
    """({name: value}, {name: bound}) of out, lse, dq, dk, dv and dbias."""
    q, k, v, dout = (O._f64(x) for x in (q, k, v, dout))
    T, H, d = q.shape
    G = H // k.shape[1]
    vals = dict(zip(("out", "lse", "dq", "dk", "dv", "dbias"), O.scored_attention(q, k, v, cu, scale, s, dout)))
    tol = {n: None if x is None else np.zeros(x.shape) for n, x in vals.items()}
    for i in range(len(cu) - 1):
        rows = slice(cu[i], cu[i + 1])
        m = cu[i + 1] - cu[i]
        if m == 0:
            continue
        prefix = s.prefix_lens[i] if len(s.prefix_lens) else 0
        for h in range(H):
            hk = h // G
            qh, kh, vh, do = q[rows, h], k[rows, hk], v[rows, hk], dout[rows, h]
            x, t, seen, dist = O._sample_scores(qh, kh, scale, s, h, prefix)
            p, lse = O._softmax(x, seen)
            mags = np.abs(x)
            if s.slopes is not None:
                mags = mags + 2 * float(O._f64(s.slopes)[h]) * np.abs(dist)
            delta = (d + 16) * U * scale * (np.abs(qh) @ np.abs(kh).T) + 4e-6 * mags
            delta = np.where(seen, delta, 0.0).max(1, initial=0.0)
            e = (2 * delta + 2.0 ** -20)[:, None]
            A = p @ np.abs(vh)
            o = p @ vh
            tol["out"][rows, h] = (r_op + e + m * U) * A + r_out * np.abs(o)
            tol["lse"][h, rows] = np.where(np.isfinite(lse), delta + 2.0 ** -20 + 2 * U * np.abs(lse), 0.0)
            eD = (np.abs(do) * (r_op + e + 2.0 ** -16 + m * U) * A).sum(1, keepdims=True)
            g = do @ vh.T - (do * o).sum(1, keepdims=True)
            w = 1.0 if t is None else 1 - t * t
            raw = np.abs(p * g)
            part = p * (eD + d * U * (np.abs(do) @ np.abs(vh).T))
            eS = (r_op + 2 * e + 4e-6) * raw * w + part + 4e-6 * raw
            eS = eS + ds_floor * seen
            mag = raw * w
            tol["dq"][rows, h] = scale * (eS @ np.abs(kh) + m * U * (mag @ np.abs(kh)))
            tol["dk"][rows, hk] += scale * (eS.T @ np.abs(qh) + G * m * U * (mag.T @ np.abs(qh)))
            tol["dv"][rows, hk] += (r_op + 2 * e.max() + G * m * U) * (p.T @ np.abs(do))
            if s.bias is not None:
                far = np.asarray(s.buckets)[np.minimum(np.abs(dist), len(s.buckets) - 1)]
                eB = (2 * e + 4e-6 + (r_op if t is not None else 0.0) + m * U) * raw + part
                np.add.at(tol["dbias"][h], far.ravel(), eB.ravel())
    return vals, tol


def check(name, got, want, tol, extra=0.0):
    """|got - want| within the bound (plus `extra` of the value), infinities in the same places."""
    got = O._f64(got)
    assert got.shape == want.shape, name
    fin = np.isfinite(want)
    assert np.array_equal(got[~fin], want[~fin]), name + ": non-finite values differ"
    err = np.abs(got[fin] - want[fin])
    lim = tol[fin] + extra * np.abs(want[fin]) + 1e-30
    assert np.all(np.isfinite(got[fin])), name + ": non-finite values"
    assert np.all(err <= lim), "%s: %.3g of the bound" % (name, float((err / lim).max()))
