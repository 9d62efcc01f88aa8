"""fp64 oracle of linear attention with a decay per head (numpy, token by token).

Per sequence and head: S_t = exp(g_t) S_{t-1} + k_t v_t^T, o_t = S_t^T q_t.

Next to each result stands a bound on what the product path's arithmetic can do to it.  Every
result is a sum of products of inputs, and the bound is relative to the sum of their magnitudes,
which the same recurrences give from |q|, |k|, |v|, |do| and the states' magnitudes:

* `u`, a rounding of a factor to the element type (2^-8 for bf16, 0 for fp32, half a step): the
  scores or the state in o, dq, dk and dv; both states in dg;
* the states themselves: u^2 at most (three terms of that type), and fp32 sums;
* fp32: every decay is a product of at most one factor per chunk and of a chunk's sum of
  log-decays, off by 4 U32 and U32 of its exponent each, and where that exponent is beyond 150 the
  term is nothing; sums over the channels and over a chunk's 64 tokens.
"""

from __future__ import annotations

import numpy as np

U32 = 2.0 ** -24


def spans(N, T, cu):
    if cu is None:
        return [(n, 0, T) for n in range(N)]
    return [(0, int(a), int(z)) for a, z in zip(cu[:-1], cu[1:])]


def _fp32(n, channels):
    """Relative error of fp32 arithmetic over n tokens: decays, sums."""
    return U32 * (8 * (n // 32 + 4) + 300 + channels + 2 * 64 + n // 32)


def la_forward(q, k, v, g, s0=None, cu=None, u=0.0):
    """(o, final state, bound on o, bound on the final state); g [B, H, T] or [H]."""
    B, H, T, dk = q.shape
    dv = v.shape[3]
    g = np.broadcast_to(g[None, :, None], (B, H, T)) if g.ndim == 1 else g
    sp = spans(B, T, cu)
    o, eo = np.zeros((B, H, T, dv)), np.zeros((B, H, T, dv))
    sf = np.zeros((len(sp), H, dk, dv)) if s0 is None else s0.copy()
    ef = np.zeros_like(sf)
    for n, (b, lo, hi) in enumerate(sp):
        S, A = sf[n].copy(), np.abs(sf[n])
        e32 = _fp32(hi - lo, dk)
        for t in range(lo, hi):
            f = np.exp(g[b, :, t])[:, None, None]
            S = f * S + k[b, :, t, :, None] * v[b, :, t, None]
            A = f * A + np.abs(k[b, :, t, :, None] * v[b, :, t, None])
            o[b, :, t] = np.einsum("hk,hkv->hv", q[b, :, t], S)
            eo[b, :, t] = (u + u * u + e32) * np.einsum("hk,hkv->hv", np.abs(q[b, :, t]), A)
        sf[n], ef[n] = S, (u * u + e32) * A
    return o, sf, eo, ef


def la_backward(q, k, v, g, do, s0=None, df=None, cu=None, u=0.0):
    """((dq, dk, dv, dg, ds0), their bounds); dg [H] where g is."""
    B, H, T, dk = q.shape
    dv = v.shape[3]
    fixed = g.ndim == 1
    g = np.broadcast_to(g[None, :, None], (B, H, T)) if fixed else g
    sp = spans(B, T, cu)
    zero = np.zeros((len(sp), H, dk, dv))
    s0, df = zero if s0 is None else s0, zero if df is None else df
    out = [np.zeros_like(q), np.zeros_like(k), np.zeros_like(v), np.zeros((B, H, T)), zero.copy()]
    err = [np.zeros_like(x) for x in out]
    for n, (b, lo, hi) in enumerate(sp):
        e32 = _fp32(hi - lo, dk + dv)
        e = u + u * u + e32
        f = np.exp(g[b, :, lo:hi])
        S, A = [s0[n]], [np.abs(s0[n])]  # before each token
        for t in range(lo, hi):
            ft, kv = f[:, t - lo, None, None], k[b, :, t, :, None] * v[b, :, t, None]
            S.append(ft * S[-1] + kv)
            A.append(ft * A[-1] + np.abs(kv))
        M, W = df[n].copy(), np.abs(df[n])
        for t in range(hi - 1, lo - 1, -1):
            i = t - lo
            qd = q[b, :, t, :, None] * do[b, :, t, None]
            M, W = M + qd, W + np.abs(qd)
            out[0][b, :, t] = np.einsum("hkv,hv->hk", S[i + 1], do[b, :, t])
            err[0][b, :, t] = e * np.einsum("hkv,hv->hk", A[i + 1], np.abs(do[b, :, t]))
            out[1][b, :, t] = np.einsum("hkv,hv->hk", M, v[b, :, t])
            err[1][b, :, t] = e * np.einsum("hkv,hv->hk", W, np.abs(v[b, :, t]))
            out[2][b, :, t] = np.einsum("hkv,hk->hv", M, k[b, :, t])
            err[2][b, :, t] = e * np.einsum("hkv,hk->hv", W, np.abs(k[b, :, t]))
            ft = f[:, i, None, None]
            out[3][b, :, t] = (ft * M * S[i]).sum((1, 2))
            # sums over a chunk's tokens and over all channels of both states
            err[3][b, :, t] = (2 * e + u * u + (64 + dk * dv // 16) * U32) * (ft * W * A[i]).sum((1, 2))
            M, W = ft * M, ft * W
        out[4][n], err[4][n] = M, (u * u + e32) * W
        if not fixed:
            # writes before a token are the chunk's less those from it on: sums that cancel
            for t0 in range(lo, hi, 32):
                part = err[3][b, :, t0:min(t0 + 64, hi)]
                err[3][b, :, t0:min(t0 + 32, hi)] += 64 * U32 * part.max(1, keepdims=True) / max(e, U32)
    if fixed:
        out[3], err[3] = out[3].sum((0, 2)), err[3].sum((0, 2)) + U32 * np.abs(out[3]).sum((0, 2))
    return out, err


def la_decode_step(q, k, v, g, S):
    """(o, S) after one token; g [N, H] or [H]."""
    f = np.exp(np.broadcast_to(g, q.shape[:2]))[..., None, None]
    S = f * S + k[..., None] * v[..., None, :]
    return np.einsum("nhk,nhkv->nhv", q, S), S
