"""fp64 oracle of softmax attention and of the 4-bit cache's format (numpy).

Next to each attention output stands a bound on what the product path's arithmetic can do to it:
fp32 scores, exponentials and sums, and weights rounded to bf16 where `weights_u` says so.
"""

from __future__ import annotations

import numpy as np

U32 = 2.0 ** -24
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def attend(q, k, v, scale, mask, weights_u):
    """One head: q [m, D], k, v [n, D], mask [m, n] (True: seen).  Returns (o, lse, bound on o,
    bound on lse); a row that sees nothing has o = 0 and lse = -inf.

    A score is a sum of D products in fp32 (an error of at most (D + 2) U32 of the sum of their
    magnitudes), times the scale; its exponential's argument is rounded once more, relative to
    the score and to the running maximum.  A weight's relative error is that error, twice (its
    own and its share of the sum), the exponential's own (4 U32) and weights_u; the sum over n
    weighted values in fp32 adds (n + 8) U32 at most."""
    m, n, D = q.shape[0], k.shape[0], q.shape[1]
    if n == 0 or m == 0:
        return np.zeros((m, v.shape[1])), np.full(m, -np.inf), np.zeros((m, v.shape[1])), np.zeros(m)
    s = scale * (q @ k.T)
    mag = abs(scale) * (np.abs(q) @ np.abs(k).T)
    s = np.where(mask, s, -np.inf)
    top = s.max(1, keepdims=True)
    safe = np.where(np.isfinite(top), top, 0.0)
    p = np.exp(s - safe)
    tot = p.sum(1, keepdims=True)
    some = tot > 0
    w = p / np.where(some, tot, 1.0)
    lse = np.where(some, safe + np.log(np.where(some, tot, 1.0)), -np.inf)[:, 0]
    err = np.where(mask, (D + 2) * U32 * mag + 4 * U32 * (np.abs(np.where(mask, s, 0.0)) + np.abs(safe)), 0.0)
    worst = err.max(1, keepdims=True)
    absum = w @ np.abs(v)
    # an exponential below fp32's range is flushed to zero: 2^-126 of the largest
    bound = absum * (2 * worst + 8 * U32 + weights_u + (n + 8) * U32) + n * 2.0 ** -126 * np.abs(v).max(initial=0.0)
    return w @ v, lse, bound, worst[:, 0] + (n + 8) * U32 + 8 * U32 * np.abs(np.where(some[:, 0], lse, 0.0))


def quantise(x):
    """x [..., D] -> (codes [..., D] 0..15, scales [..., D/32] bytes)."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    top = np.abs(b).max(-1)
    e = np.full(top.shape, -126)
    big = top > 0
    e[big] = np.maximum(np.floor(np.log2(top[big])).astype(int) - 2, -126)
    y = np.abs(b) * 2.0 ** -e[..., None]
    # the nearest magnitude; where two are as near, the one with the even code
    far = np.abs(y[..., None] - E2M1)
    code = np.argmin(far, -1)
    up = np.minimum(code + 1, 7)
    tie = np.take_along_axis(far, code[..., None], -1) == np.take_along_axis(far, up[..., None], -1)
    code = np.where(tie[..., 0] & (code % 2 == 1), up, code)
    code = code + 8 * (b < 0)
    return code.reshape(x.shape), (e + 127).astype(np.uint8)


def values(codes, scales):
    table = np.concatenate([E2M1, -E2M1])
    s = 2.0 ** (scales.astype(np.float64) - 127)
    return (table[codes].reshape(*codes.shape[:-1], -1, 32) * s[..., None]).reshape(codes.shape)
