"""Attention over local positions in 64 bits, joined and turned, with the bounds of a kernel's error. Imported by tests
only."""
from __future__ import annotations

import numpy as np

import rows_ref


def entries(t, n_vis, max_n, rows, window=0, group=1, **where):
    """Cache rows that query t sees, one by one from the definition"""
    n = min(max(int(n_vis[t]), 0), max_n)
    run = t // group
    where = {k: (v[run:run + 1] if k in ("kv_base", "seq") and v is not None else v) for k, v in where.items()}
    if where.get("pages") is not None and where.get("seq") is None:
        where["seq"] = [run]
    found = []
    for p in range(max(0, n - window) if window else 0, n):
        r = rows_ref.row_of(0, [p], max_n, rows, **where)
        if r >= 0:
            found.append(r)
    return found


def query(q, kv, scale, other=None, other_lse=None, turn=None):
    """One query: q [heads, 512] over rows kv [n, 512] (64 bits) -> (out, lse, bound of out, bound of lse). turn:
    (position, freq, offset, layout, mscale)."""
    heads, n = len(q), len(kv)
    if n:
        s = scale * (q @ kv.T)
        top = s.max(1, keepdims=True)
        e = np.exp(s - top)
        z = e.sum(1, keepdims=True)
        p = e / z
        o, l = p @ kv, (top + np.log(z))[:, 0]
        # Logits: 512 fp32 additions in any order, 2^-24 each, of terms that sum to B, and the product with scale; the
        # exponential 2^-22 and 2^-22 of the logit. In a probability and in the sum. Probabilities in 11 bits: 2^-11 of A.
        # n additions of p kv and of the sum, 2^-24 each; those of parts, lanes and wavefronts, 64 + 25. Probabilities
        # below 2^-20 of the largest: half a step of fp16's smallest numbers, 2^-31 of it, each.
        B = (abs(scale) * (np.abs(q) @ np.abs(kv).T)).max(1)
        logit = 513 * 2.0 ** -24 * B + 2.0 ** -22 + np.abs(s).max(1) * 2.0 ** -22
        adds = (n + 89) * 2.0 ** -24
        eo = (p @ np.abs(kv)) * (2.0 ** -11 + 2 * logit + 2 * adds + 2.0 ** -21)[:, None] + 2.0 ** -31 * np.abs(kv).sum(0)
        el = logit + adds + 2.0 ** -22 + 2.0 ** -22 * np.abs(l)
    else:
        o, l = np.zeros((heads, 512)), np.full(heads, -np.inf)
        eo, el = np.zeros((heads, 512)), np.zeros(heads)
    if other is not None:
        both = np.logaddexp(l, other_lse)
        with np.errstate(invalid="ignore"):
            w1 = np.where(np.isneginf(l), 0.0, np.exp(l - both))
            w2 = np.where(np.isneginf(other_lse), 0.0, np.exp(other_lse - both))
        other = np.where((w2 > 0)[:, None], other, 0.0)
        # of the weights: the logarithms' errors and differences (2^-22 of either), exponentials and quotient 2^-20
        size = np.maximum(np.abs(np.where(np.isfinite(l), l, 0)), np.abs(np.where(np.isfinite(other_lse), other_lse, 0)))
        ew = el + 2.0 ** -20 + size * 2.0 ** -21
        sizes = w1[:, None] * np.abs(o) + w2[:, None] * np.abs(other)
        eo = w1[:, None] * eo + sizes * ew[:, None]
        o = w1[:, None] * o + w2[:, None] * other
        el, l = ew + 2.0 ** -22 * np.abs(np.where(np.isfinite(both), both, 0)), both
    if turn is not None:
        pos, freq, offset, layout, m = turn
        h = len(freq)
        i0 = offset + (np.arange(h) if layout == "half" else 2 * np.arange(h))
        i1 = i0 + (h if layout == "half" else 1)
        size = np.abs(o)
        # the angle 2^-23 rad and its rounding, sin and cos, factor, products and sum: 2^-20 of |x0| + |x1|
        pair = eo[:, i0] + eo[:, i1] + 2.0 ** -20 * (size[:, i0] + size[:, i1])
        o = rows_ref.rotate(o, np.full(heads, pos), freq, offset, layout, m, inverse=True)
        eo = eo.copy()
        eo[:, i0] = eo[:, i1] = m * pair
    return o, l, eo * (1 + 2.0 ** -7) + 2.0 ** -8 * np.abs(o), el
