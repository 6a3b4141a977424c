"""References in 64 bits for the attention-side operators, from their definitions. Imported by tests only."""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


def e4m3(b: np.ndarray) -> np.ndarray:
    b = b.astype(np.int64)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e - 7.0))
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b & 128, -v, v)


def kv_rows(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """[m, 256], [m, 32] -> fp64 [m, 512]"""
    v = np.stack([E2M1[codes & 15], E2M1[codes >> 4]], -1).reshape(len(codes), 512)
    return v * np.repeat(e4m3(scales), 16, axis=1)


def entries(t, n_vis, max_n, rows, kv_base=None, pages=None, page_size=0, seq=None, idx=None, window=0):
    """(slots, cache rows) of query t: the definition's entries, one by one"""
    n = min(max(int(n_vis[t]), 0), max_n)
    pos = [(i, int(p)) for i, p in enumerate(idx[t])] if idx is not None else \
        [(p, p) for p in range(max(0, n - window) if window else 0, n)]
    slots, where = [], []
    for i, p in pos:
        if p < 0 or p >= n:
            continue
        if pages is not None:
            s = int(seq[t]) if seq is not None else t
            if s < 0 or s >= len(pages) or pages[s][p // page_size] < 0:
                continue
            r = int(pages[s][p // page_size]) * page_size + p % page_size
        else:
            r = int(kv_base[t]) + p
        if 0 <= r < rows:
            slots.append(i)
            where.append(r)
    return slots, where


def attention(q, codes, scales, scale, where):
    """One query: q [heads, 512] fp64 over the rows `where` -> dict with out, lse, p, and the magnitudes the
    tolerances are relative to: A = sum p |kv|, B = largest scale * sum |q| |kv| of any (head, entry)."""
    heads = len(q)
    if not where:
        return dict(out=np.zeros((heads, 512)), lse=np.full(heads, -np.inf), p=np.zeros((heads, 0)),
                    s=np.zeros((heads, 0)), A=np.zeros((heads, 512)), B=0.0)
    kv = kv_rows(codes[where], scales[where])
    s = scale * (q @ kv.T)
    m = s.max(1, keepdims=True)
    e = np.exp(s - m)
    z = e.sum(1, keepdims=True)
    p = e / z
    return dict(out=p @ kv, lse=(m + np.log(z))[:, 0], p=p, s=s, A=p @ np.abs(kv),
                B=float((abs(scale) * (np.abs(q) @ np.abs(kv).T)).max()))


def out_tolerance(r, n):
    """bf16 result, half a step: 2^-8 |o|. Probabilities in 11 bits: 2^-11 A. Logits: 512 fp32 additions in any
    order, 2^-24 each, of terms that sum to B, and the product with scale: 513 * 2^-24 B, in the probability and
    in the sum; their exponential, 2^-22 relative and |s| 2^-23 of the base-2 logit. n fp32 additions of p kv and
    of the sum. A probability below 2^-20 of the largest is off by
    up to half a step of fp16's smallest numbers, 2^-25 where the largest is above 2^6: 2^-31 of it, n times."""
    big = np.abs(r["s"]).max(initial=0.0)
    rel = 2.0 ** -11 + 2 * (513 * 2.0 ** -24 * r["B"] + 2.0 ** -22 + big * 2.0 ** -22) + 2 * n * 2.0 ** -24
    return 2.0 ** -8 * np.abs(r["out"]) + r["A"] * rel + n * 2.0 ** -31 * 2688


def lse_tolerance(r, n):
    big = np.abs(r["s"]).max(initial=0.0)
    return 513 * 2.0 ** -24 * r["B"] + (big + 1) * 2.0 ** -22 + n * 2.0 ** -24 + np.abs(r["lse"]) * 2.0 ** -23


def weight_tolerance(r, w):
    big = np.abs(r["s"]).max(initial=0.0)
    return w * 1.05 * (513 * 2.0 ** -24 * r["B"] + (big + 4) * 2.0 ** -21)
