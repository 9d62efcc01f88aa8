"""fp64 oracle of attention weights per cached token, and of eviction by them (numpy)."""

from __future__ import annotations

import numpy as np

from .attn_oracle import U32


def weigh(q, k, lse, scale, mask):
    """One head: the weight that queries q [m, D] give to keys k [n, D], mask [m, n] (True: seen),
    and its bound: the score's fp32 sum and product, the exponent's two roundings (relative to
    the score and to lse), the exponential's own and m additions."""
    m, D = q.shape
    if m == 0 or k.shape[0] == 0:
        return np.zeros(k.shape[0]), np.zeros(k.shape[0])
    use = mask & np.isfinite(lse)[:, None]
    s = scale * (q @ k.T)
    base = np.where(np.isfinite(lse), lse, 0.0)[:, None]
    p = np.where(use, np.exp(np.where(use, s - base, 0.0)), 0.0)
    mag = abs(scale) * (np.abs(q) @ np.abs(k).T)
    err = p * ((D + 2) * U32 * mag + 4 * U32 * (np.abs(s) + np.abs(base)) + 8 * U32)
    return p.sum(0), err.sum(0) + (m + 8) * U32 * p.sum(0) + m * 2.0 ** -126


def evict(weights, length, budget, recent):
    """Positions that stay, in order, of one head's tokens with weights [length]."""
    if length <= budget:
        return np.arange(length)
    free = length - recent
    w = np.where(np.isnan(weights[:free]), np.inf, weights[:free])
    nan = np.isnan(weights[:free])
    order = np.lexsort((np.arange(free), -w, ~nan))
    return np.concatenate([np.sort(order[:budget - recent]), np.arange(free, length)])
