"""Attention whose queries are cut into parts that are joined, over caches that show which entries were taken: one token
over long ranges and batches in unequal numbers of parts. Within the bounds of attn_bounds.py, which see a single step."""
import numpy as np
import pytest
import torch

import attn_bounds as ab
import attn_ref as ref

pytestmark = pytest.mark.gpu
SCALE = 512 ** -0.5


@pytest.fixture(scope="module")
def fx():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import top_fp4_lightning_amd

    return top_fp4_lightning_amd


def dev(a, dt):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=dt)).cuda()


def run(fx, q, codes, scales, nv, n, entries, **where):
    nq, heads = q.shape[:2]
    out, lse = torch.empty(nq, heads, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(nq, heads, device="cuda")
    fx.idx_attend(torch.from_numpy(q).bfloat16().cuda(), dev(codes, np.uint8), dev(scales, np.uint8), dev(nv, np.int32), n,
                  SCALE, out, fx.workspace(fx.IDX_OP_ATTEND, nq, entries, heads), lse=lse, **where)
    torch.cuda.synchronize()
    return out.double().cpu().numpy(), lse.double().cpu().numpy()


def compare(fx, got, q, codes, scales, queries, entries):
    """queries: t -> its entries (rows of codes, scales), in order"""
    parts = ab.parts_of(fx, *q.shape[:2], entries)
    for t, where in queries.items():
        r = ref.attention(q[t].astype(np.float64), codes, scales, SCALE, where)
        if not where:
            assert (got[0][t] == 0).all() and np.isneginf(got[1][t]).all(), t
            continue
        out_tol, lse_tol = ab.bounds(r, ref.kv_rows(codes[where], scales[where]), parts, entries)
        err = np.abs(got[0][t] - r["out"])
        assert (err <= out_tol).all(), (t, err.max(), np.argwhere(err > out_tol)[:3])
        assert (np.abs(got[1][t] - r["lse"]) <= lse_tol).all(), (t, np.abs(got[1][t] - r["lse"]).max())


@pytest.mark.parametrize("nq,heads,n", ab.CASES)
def test_every_step_counts(fx, nq, heads, n):
    """contiguous, in pages that end inside a step, and as a list in any order"""
    q, nv, long, rng = ab.case(nq, heads, n)
    codes, scales = ab.marked_rows(rng, n)
    some = sorted({*long, *range(1, nq, max(1, nq // 8))})
    print(f"attend long nq={nq} heads={heads} n={n} parts={ab.parts_of(fx, nq, heads, n)}", flush=True)
    queries = {t: list(range(nv[t])) for t in some}
    compare(fx, run(fx, q, codes, scales, nv, n, n, kv_base=dev(np.zeros(nq), np.int64)), q, codes, scales, queries, n)
    page = 24
    per = -(-n // page)
    order = rng.permutation(per + 2)[:per]
    rows = order[np.arange(n) // page] * page + np.arange(n) % page
    paged = rng.integers(0, 256, ((per + 2) * page, 256), dtype=np.uint8), np.full(((per + 2) * page, 32), 0x7F, np.uint8)
    paged[0][rows], paged[1][rows] = codes, scales
    got = run(fx, q, *paged, nv, n, n, pages=dev(order[None], np.int32), page_size=page, seq=dev(np.zeros(nq), np.int32))
    compare(fx, got, q, codes, scales, queries, n)
    perm = rng.permutation(n)
    mixed = np.empty_like(codes), np.empty_like(scales)
    mixed[0][perm], mixed[1][perm] = codes, scales
    idx = np.where(np.arange(n) < nv[:, None], perm, -1)
    got = run(fx, q, *mixed, np.full(nq, n), n, n, kv_base=dev(np.zeros(nq), np.int64), idx=dev(idx, np.int32))
    compare(fx, got, q, codes, scales, queries, n)


@pytest.mark.parametrize("window", [1, 63, 64, 65, 128, 1000, 5000])
@pytest.mark.parametrize("page", [1, 24, 64, 100])
def test_windows_in_pages(fx, page, window):
    """windows that begin inside a page and end inside one, of more than one part, over pages of mixed order"""
    rng = np.random.default_rng(window + page)
    n = 6000
    codes, scales = ab.marked_rows(rng, n)
    per = -(-n // page)
    order = np.stack([rng.permutation(per + 3)[:per] for _ in range(1)])
    rows = order[0][np.arange(n) // page] * page + np.arange(n) % page
    total = (per + 3) * page
    paged = rng.integers(0, 256, (total, 256), dtype=np.uint8), np.full((total, 32), 0x7F, np.uint8)
    paged[0][rows], paged[1][rows] = codes, scales
    nv = np.array([n, n - 1, 4097, window, max(window - 1, 0), 1, 0, n - 77])
    q = rng.standard_normal((len(nv), 20, 512)).astype(np.float32)
    q = (q.view(np.uint32) & 0xFFFF0000).view(np.float32)
    print(f"attend window={window} page={page}", flush=True)
    got = run(fx, q, *paged, nv, n, window, pages=dev(order, np.int32), page_size=page, seq=dev(np.zeros(len(nv)), np.int32),
              window=window)
    compare(fx, got, q, codes, scales, {t: list(range(max(0, m - window), m)) for t, m in enumerate(nv)}, window)
