"""fp64 oracle of the gated linear recurrence (numpy, token by token).

Per sequence, head and channel: h_t = exp(g_t) h_{t-1} + x_t, o_t = h_t.  The backward takes
the forward's outputs as it is given them (rounded or not) for h_{t-1}.

Next to each result stands a bound on what fp32 arithmetic can do to it, whatever the order in
which the affine maps y -> exp(g) y + x are composed: every decay that a value passes brings a
relative error of at most `decay_err(g)`, every addition one rounding of the running sum of
magnitudes.
"""

from __future__ import annotations

import numpy as np

U32 = 2.0 ** -24  # a rounding to fp32, relative


def decay_err(g):
    """Relative error of one computed factor exp(g) and of the product it enters: the
    hardware's exponential (2 U32), its argument's rounding (2 U32 |g|) and the product's own
    rounding (U32), with one more for the factor's place in a product of factors."""
    return U32 * (4.0 + 2.0 * np.minimum(np.abs(g), 200.0))


def _spans(N, T, cu):
    if cu is None:
        return [(n, 0, T) for n in range(N)]
    return [(0, int(a), int(z)) for a, z in zip(cu[:-1], cu[1:])]


def _scan(a, x, y0, err):
    """y_t = a_t y_{t-1} + x_t over axis 1 of [H, T, d]; returns all y, and their fp32 bound."""
    y, mag, e = y0.copy(), np.abs(y0), np.zeros_like(y0)
    ys, es = np.empty_like(x), np.empty_like(x)
    for t in range(x.shape[1]):
        e = a[:, t] * (e + err[:, t] * mag)
        y = a[:, t] * y + x[:, t]
        mag = a[:, t] * mag + np.abs(x[:, t])
        e = e + 2 * U32 * mag
        ys[:, t], es[:, t] = y, e
    return ys, es


def glr_forward(x, g, h0=None, cu=None):
    """(o, final state, bound on o, bound on the final state), all fp64."""
    B, H, T, d = x.shape
    spans = _spans(B, T, cu)
    h0 = np.zeros((len(spans), H, d)) if h0 is None else h0
    o, bound = np.zeros_like(x), np.zeros_like(x)
    hf, bf = h0.copy(), np.zeros_like(h0)
    for n, (b, lo, hi) in enumerate(spans):
        if hi > lo:
            o[b, :, lo:hi], bound[b, :, lo:hi] = _scan(np.exp(g[b, :, lo:hi]), x[b, :, lo:hi], h0[n],
                                                       decay_err(g[b, :, lo:hi]))
            hf[n], bf[n] = o[b, :, hi - 1], bound[b, :, hi - 1]
    return o, hf, bound, bf


def glr_backward(g, o, do, h0=None, dfinal=None, cu=None):
    """(dx, dg, dh0) and the bound on each."""
    B, H, T, d = g.shape
    spans = _spans(B, T, cu)
    zero = np.zeros((len(spans), H, d))
    h0, dfinal = zero if h0 is None else h0, zero if dfinal is None else dfinal
    dx, dg, ex, eg = (np.zeros_like(g) for _ in range(4))
    d0, e0 = dfinal.copy(), zero.copy()
    for n, (b, lo, hi) in enumerate(spans):
        if hi == lo:
            continue
        a, do_n = np.exp(g[b, :, lo:hi]), do[b, :, lo:hi]
        prev = np.concatenate([h0[n][:, None], o[b, :, lo:hi - 1]], 1)
        # the gradient that reaches h_{t-1}, last token first: e_t = a_t (do_t + e_{t+1})
        e, mag, err = dfinal[n].copy(), np.abs(dfinal[n]), np.zeros_like(h0[n])
        for t in range(hi - lo - 1, -1, -1):
            dh, mag = do_n[:, t] + e, mag + np.abs(do_n[:, t])
            err = err + 2 * U32 * mag
            dx[b, :, lo + t], ex[b, :, lo + t] = dh, err
            err = a[:, t] * (err + decay_err(g[b, :, lo + t]) * mag)
            e, mag = a[:, t] * dh, a[:, t] * mag
            dg[b, :, lo + t] = e * prev[:, t]
            eg[b, :, lo + t] = (err + 2 * U32 * mag) * np.abs(prev[:, t])
        d0[n], e0[n] = e, err + 2 * U32 * mag
    return dx, dg, d0, ex, eg, e0


def glr_decode_step(x, g, h):
    return np.exp(g) * h + x
