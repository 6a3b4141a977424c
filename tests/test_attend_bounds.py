"""The bounds of attn_bounds.py see what they are for (no GPU): the definition without one step of 64 entries, or without
one part of a query's entries, or with the last entries missing, lies outside them."""
import numpy as np
import pytest

import attn_bounds as ab
import attn_ref as ref
from test_abi import fx  # noqa: F401

SCALE = 512 ** -0.5


@pytest.mark.parametrize("nq,heads,n", ab.CASES)
def test_a_missing_step_or_part_is_seen(fx, nq, heads, n):
    q, nv, long, rng = ab.case(nq, heads, n)
    codes, scales = ab.marked_rows(rng, n)
    parts = ab.parts_of(fx, nq, heads, n)
    for t in long[:2] + long[-1:]:
        m = int(nv[t])
        r = ref.attention(q[t].astype(np.float64), codes, scales, SCALE, list(range(m)))
        kv = ref.kv_rows(codes[:m], scales[:m])
        out_tol, lse_tol = ab.bounds(r, kv, parts, n)
        i = np.arange(m)
        steps = -(-m // 64)
        lost = [i // 64 == s for s in range(steps)] if m > 64 else []
        for k in {*parts} - {1}:
            per = -(-steps // k)
            lost += [i // (64 * per) == s for s in range(-(-steps // per))]
        lost += [i == m - 1, i == 0, i % 64 == 63]
        for gone in lost:
            if gone.all():
                continue
            out, lse = ab.without(r, kv, gone)
            # in every head: by the output alone
            assert (np.abs(out - r["out"]) > out_tol).any(1).all(), (t, gone.nonzero()[0][:2])
        for gone in lost[:steps if m > 64 else 0]:
            _, lse = ab.without(r, kv, gone)
            assert (np.abs(lse - r["lse"]) > lse_tol).all(), t
        zeros = np.abs(r["out"]) > out_tol
        used = np.abs(kv).sum(0) > 0
        assert zeros[:, used].mean() > 0.95, zeros[:, used].mean()  # an output of zeros is no pass


def test_parts_of_a_call(fx):
    assert ab.parts_of(fx, 1, 64, 64) == (1, 1)
    low, high = ab.parts_of(fx, 514, 64, 16384)
    assert 1 <= low < high == low + 1
