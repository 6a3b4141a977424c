"""Caches that show which entries an attention call took, and bounds tight enough to see a step or a part of them
missing, taken twice or joined wrongly. Imported by tests only."""
from __future__ import annotations

import numpy as np

import attn_ref as ref

STEP = 64           # entries of a step
MOST = 320 * STEP   # entries that the marks tell apart


def marked_rows(rng, n):
    """Codes and scales of entries 0 .. n - 1 (n <= MOST). Value i // 64 is 6 and so is value 448 + i % 64, which mark an
    entry's step and its place in it; values 320 .. 447 are random, the others zero."""
    assert n <= MOST
    v = np.zeros((n, 512), np.uint8)
    v[:, 320:448] = rng.integers(0, 16, (n, 128))
    i = np.arange(n)
    v[i, i // STEP] = 7
    v[i, 448 + i % STEP] = 7
    codes = v[:, 0::2] | (v[:, 1::2] << 4)
    scales = np.full((n, 32), 0x38, np.uint8)
    scales[:, 20:28] = rng.integers(0x18, 0x2C, (n, 8))
    return codes, scales


def parts_of(fx, nq, heads, entries):
    """(fewest, most) parts that a query's entries are cut into, from the size of the call's workspace: 514 fp32 for
    each head of each part"""
    size = fx.workspace_size(fx.IDX_OP_ATTEND, nq, entries, heads)
    if size == 16:
        return 1, 1
    units, rest = divmod(size, heads * 514 * 4)
    assert rest == 0
    return units // nq, -(-units // nq)


def bounds(r, kv, parts, entries):
    """Of (out, lse) for a query with rows kv [n, 512] (64 bits) in a call of `entries` entries cut into between
    parts[0] and parts[1] parts.

    out: half a step of bf16, 2^-8 of it. Relative to A = sum p |kv|: probabilities in 11 bits, 2^-11; logits, in the
    probability and in the sum: 512 additions and the product with scale, 2^-24 each of B, and the exponential, 2^-22
    and 2^-22 of the logit; the reciprocal and its product 2^-22; one rounding for each addition: of a value, those of
    entries that are not zero there (adding zero is exact, as is moving the reference by powers of two) and one per
    part; of the sum, four and one for a step, one per part and 25 over lanes and wavefronts. Probabilities below 2^-20
    of the largest are off by half a step of fp16's smallest numbers, 2^-31 of it.
    lse: the logits' and the sum's part of that, its logarithm and result 2^-23 of it and 2^-22."""
    n = len(kv)
    big, steps = np.abs(r["s"]).max(initial=0.0), -(-entries // STEP)
    sums = 4 + -(-steps // parts[0]) + parts[1] + 25
    logit = 513 * 2.0 ** -24 * r["B"] + 2.0 ** -22 + big * 2.0 ** -22
    adds = np.minimum((kv != 0).sum(0), -(-steps // parts[0]) * STEP) + parts[1]
    rel = 2.0 ** -11 + 2 * logit + 2.0 ** -22 + (adds + sums) * 2.0 ** -24
    out = 2.0 ** -8 * np.abs(r["out"]) + r["A"] * rel + 2.0 ** -31 * np.abs(kv).sum(0)
    lse = logit + 2.0 ** -22 + sums * 2.0 ** -24 + 2.0 ** -23 * np.abs(r["lse"])
    return out, lse


def without(r, kv, gone):
    """(out, lse) of the same query without the entries of the mask `gone` [n]"""
    p = r["p"][:, gone]
    left = 1.0 - p.sum(1, keepdims=True)
    return (r["out"] - p @ kv[gone]) / left, r["lse"] + np.log(left[:, 0])


# (queries, heads, longest): one token over a long range, and batches whose queries are cut into unequal numbers of parts
CASES = [(2, 3, 20011), (1, 64, 20480), (300, 2, 1000), (300, 40, 4096), (200, 16, 9000), (300, 20, 6000), (90, 64, 12000),
         (600, 5, 3000), (700, 16, 2000)]


def case(nq, heads, n):
    """(q as bf16 values, n_vis, long queries): most queries short, a few of (nearly) full length on both sides of the
    places where the number of parts may change"""
    rng = np.random.default_rng(nq + heads + n)
    q = rng.standard_normal((nq, heads, 512)).astype(np.float32)
    q = (q.view(np.uint32) & 0xFFFF0000).view(np.float32)
    nv = rng.integers(0, 90, nq)
    long = sorted({0, nq // 4, nq // 3, nq // 2, nq - 2 if nq > 1 else 0, nq - 1})
    nv[long] = n - rng.integers(0, 64, len(long))
    nv[0] = n
    return q, nv, long, rng
