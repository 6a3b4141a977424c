"""idx_attend_local against its definition in 64 bits (local_ref.py), within bounds counted from half-step roundings."""
import numpy as np
import pytest
import torch

import local_ref
import rows_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fx():
    import top_fp4_lightning_amd as fx

    return fx


def dev(x):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()


def bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).bfloat16().float().numpy()


def cache(rng, rows):
    y = rng.standard_normal((rows, 512)) * np.exp(rng.standard_normal((rows, 1)))
    codes, scales = rows_ref.quantise("local", y)
    return codes, scales


def where_of(kind, rng, runs, n, ring):
    """(arguments, rows of the cache)"""
    span = ring or n
    if kind == "base":
        return dict(kv_base=(rng.permutation(runs) * span + 3).astype(np.int64)), runs * span + 5
    page = {"pages": 16, "odd": 7, "one": 1}[kind]
    per = -(-span // page)
    seqs = runs + 2
    pages = rng.permutation(seqs * per).reshape(seqs, per).astype(np.int32)
    return dict(pages=pages, page_size=page, seq=rng.permutation(seqs)[:runs].astype(np.int32)), seqs * per * page


def run(fx, q, codes, scales, n_vis, max_n, scale, where, ws=None, other=None, other_lse=None, turn=None, pos=None, lse=True,
        **kw):
    nq, heads, _ = q.shape
    bf = lambda x: dev(x).bfloat16()  # noqa: E731
    out = torch.full((nq, heads, 512), 9.0, dtype=torch.bfloat16, device="cuda")
    l = torch.full((nq, heads), 9.0, device="cuda") if lse else None
    entries = min(max_n, kw["window"] + kw.get("group", 1) - 1) if kw.get("window") else max_n
    if ws is None:
        ws = torch.full((fx.workspace_size(fx.IDX_OP_ATTEND_LOCAL, nq, entries, heads),), 255, dtype=torch.uint8, device="cuda")
    tk = {} if turn is None else dict(pos=dev(pos), freq=dev(turn[0]), offset=turn[1], layout=turn[2], mscale=turn[3])
    fx.idx_attend_local(bf(q), dev(codes), dev(scales), dev(n_vis), max_n, scale, out, ws, lse=l,
                        other=None if other is None else bf(other), other_lse=dev(other_lse),
                        **{k: dev(v) if isinstance(v, np.ndarray) else v for k, v in where.items()}, **tk, **kw)
    return out.double().cpu().numpy(), None if l is None else l.double().cpu().numpy()


def check(got, q, codes, scales, n_vis, max_n, scale, where, other=None, other_lse=None, turn=None, pos=None, which=None, **kw):
    kw.pop("ring_", None)
    for t in range(len(q)) if which is None else which:
        rows = local_ref.entries(t, n_vis, max_n, len(codes), window=kw.get("window", 0), group=kw.get("group", 1),
                                 ring=kw.get("ring", 0), **where)
        o, l, eo, el = local_ref.query(q[t].astype(np.float64), rows_ref.values("local", codes[rows], scales[rows]), scale,
                                       None if other is None else other[t].astype(np.float64),
                                       None if other is None else other_lse[t].astype(np.float64),
                                       None if turn is None else (pos[t], *turn))
        assert np.array_equal(np.isneginf(l), np.isneginf(got[1][t])), t
        fin = np.isfinite(l)
        assert (np.abs(got[1][t][fin] - l[fin]) <= el[fin]).all(), (t, np.abs(got[1][t][fin] - l[fin]).max())
        assert (np.abs(got[0][t] - o) <= eo).all(), (t, (np.abs(got[0][t] - o) - eo).max())


FREQ = 10000.0 ** (-np.arange(0, 64, 2) / 64)
# runs, group, heads, n, window, kind, ring, join, turn
CASES = [
    (1, 1, 64, 131, 128, "base", True, True, (FREQ, 448, "interleaved", 0.75)),
    (3, 1, 64, 300, 128, "pages", True, True, (FREQ, 448, "half", 1.0)),
    (5, 1, 1, 40, 0, "base", False, False, None),
    (2, 7, 5, 200, 128, "odd", True, True, (FREQ[:17], 3, "half", 1.5)),
    (2, 33, 1, 90, 16, "pages", False, False, None),
    (1, 40, 16, 500, 128, "base", False, True, (FREQ, 448, "interleaved", 1.0)),
    (2, 3, 100, 65, 64, "one", True, False, (10000.0 ** (-np.arange(0, 512, 2) / 512), 0, "interleaved", 1.0)),
    (1, 2, 128, 129, 0, "odd", False, True, (10000.0 ** (-np.arange(0, 512, 2) / 512), 0, "half", 0.5)),
    (4, 2, 17, 1000, 1, "base", True, False, None),
    (1, 1, 33, 1, 128, "base", False, False, None),
    (1, 5, 64, 5, 3, "pages", True, True, None),
    (1, 1, 16, 3000, 0, "pages", False, True, (FREQ, 448, "interleaved", 1.0)),
    (2, 3, 64, 2500, 0, "odd", False, False, None),
    (1, 50, 3, 700, 0, "base", False, False, None),
    (300, 1, 2, 70, 64, "base", False, False, None),
    (1, 1, 8, 700, 600, "pages", True, False, None),
    (250, 1, 50, 90, 80, "base", False, True, (FREQ, 448, "half", 1.0)),
    (50, 4, 64, 200, 128, "odd", True, True, (FREQ[:17], 4, "interleaved", 1.5)),
    (140, 1, 32, 128, 0, "pages", False, True, (10000.0 ** (-np.arange(0, 512, 2) / 512), 0, "interleaved", 0.5)),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_against_the_definition(fx, case):
    runs, group, heads, n, window, kind, rings, join, turn = CASES[case]
    rng = np.random.default_rng(case)
    ring = window + group - 1 + (case % 3) if rings else 0
    far = 5000 if ring else 0  # a ring's entries may have any number
    where, rows = where_of(kind, rng, runs, n, ring)
    codes, scales = cache(rng, rows)
    nq = runs * group
    last = n - rng.integers(0, max(1, (n - group) // 4 + 1), runs)
    n_vis = (far + last[:, None] - group + 1 + np.arange(group)).reshape(-1).astype(np.int32)
    if nq > 3:
        n_vis[nq // 2] = 0
        n_vis[1] = -5
    max_n = far + n
    q = bf16(2 * rng.standard_normal((nq, heads, 512)))
    scale = (-1) ** case * 0.05
    other = other_lse = None
    if join:
        other = bf16(rng.standard_normal((nq, heads, 512)))
        other_lse = np.float32(3 + 3 * rng.standard_normal((nq, heads)))
        other_lse[:, 0] = -np.inf
        other[:, 0] = np.nan  # has no effect
        if nq > 3:
            other_lse[nq // 2] = -np.inf
    pos = rng.integers(0, 1 << 20, nq)
    kw = dict(window=window, ring=ring, group=group)
    got = run(fx, q, codes, scales, n_vis, max_n, scale, where, other=other, other_lse=other_lse, turn=turn, pos=pos, **kw)
    some = range(nq) if nq <= 60 else rng.choice(nq, 60, replace=False)
    check(got, q, codes, scales, n_vis, max_n, scale, where, other, other_lse, turn, pos, which=some, **kw)
    # the same again, and without the logarithms
    again = run(fx, q, codes, scales, n_vis, max_n, scale, where, other=other, other_lse=other_lse, turn=turn, pos=pos,
                lse=False, **kw)
    assert np.array_equal(again[0], got[0])


@pytest.mark.parametrize("runs, group, heads, n", [(1, 1, 3, 9000), (1, 2, 64, 5000), (7, 1, 20, 3001), (1, 4, 16, 640),
                                                   (2, 9, 64, 3000), (1, 300, 64, 4000), (2, 150, 64, 3000)])
def test_parts_of_long_ranges(fx, runs, group, heads, n):
    """entries that mark their step and their place in it, over calls in one part and in many: a missing or repeated step
    or entry moves a value by 1/64 of itself, its bound is about 2^-8"""
    rng = np.random.default_rng(n)
    v = 0.01 * rng.standard_normal((runs * n, 512))
    i = np.arange(runs * n) % n
    v[np.arange(runs * n), i // 64 % 400] = 6.0
    v[np.arange(runs * n), 400 + i % 64] = 6.0
    codes, scales = rows_ref.quantise("local", v)
    where = dict(kv_base=np.arange(runs, dtype=np.int64) * n)
    nq = runs * group
    n_vis = (n - group + 1 + np.tile(np.arange(group), runs)).astype(np.int32)
    q = bf16(0.05 * rng.standard_normal((nq, heads, 512)))
    full = run(fx, q, codes, scales, n_vis, n, 0.04, where, group=group)
    some = sorted({0, 1 % nq, nq // 3, nq // 2, max(0, nq - 2), nq - 1})  # (runs are cut into unequal numbers of parts)
    check(full, q, codes, scales, n_vis, n, 0.04, where, group=group, which=some)
    size = fx.workspace_size(fx.IDX_OP_ATTEND_LOCAL, nq, n, heads)
    assert size > 16
    for room in (16, max(16, size // 2), size + 4096):
        ws = torch.full((room,), 255, dtype=torch.uint8, device="cuda")
        got = run(fx, q, codes, scales, n_vis, n, 0.04, where, group=group, ws=ws)
        check(got, q, codes, scales, n_vis, n, 0.04, where, group=group, which=some)


@pytest.mark.parametrize("runs, group, heads, n, kind", [(64, 1, 16, 8000, "base"), (5, 2, 64, 20000, "pages"),
                                                         (33, 3, 20, 8192, "odd"), (2, 8, 128, 4097, "base")])
def test_runs_of_different_lengths(fx, runs, group, heads, n, kind):
    """long ranges whose lengths differ from run to run and within one: steps marked as above, one cache for all"""
    rng = np.random.default_rng(runs)
    page = {"base": 1, "pages": 64, "odd": 7}[kind]
    rows = n + 64 * runs + page
    v = 0.01 * rng.standard_normal((rows, 512))
    i = np.arange(rows)
    v[i, i // 64 % 400] = 6.0
    v[i, 400 + i % 64] = 6.0
    codes, scales = rows_ref.quantise("local", v)
    if kind == "base":
        where = dict(kv_base=64 * np.arange(runs, dtype=np.int64))
    else:
        pages = np.arange(runs)[:, None] * 64 // page + np.arange(-(-n // page))
        where = dict(pages=pages.astype(np.int32), page_size=page, seq=rng.permutation(runs).astype(np.int32))
    q = bf16(0.05 * rng.standard_normal((runs * group, heads, 512)))
    ws = torch.full((fx.workspace_size(fx.IDX_OP_ATTEND_LOCAL, runs * group, n, heads) + 4096,), 255, dtype=torch.uint8,
                    device="cuda")
    for lengths in ("any", "few", "alike", "none"):
        last = {"any": rng.integers(0, n + 1, runs), "few": np.full(runs, 70), "alike": np.full(runs, n),
                "none": np.zeros(runs)}[lengths].astype(np.int64)
        if lengths == "few":
            last[-1], last[0] = n, -3
        n_vis = (last[:, None] - np.arange(group)[::-1]).reshape(-1).astype(np.int32)
        if group > 2:
            n_vis[1] = n + 5
            n_vis[-2] = 0
        got = run(fx, q, codes, scales, n_vis, n, 0.04, where, group=group, ws=ws)
        some = sorted({0, 1, 2, runs * group // 2, runs * group - 2, runs * group - 1})
        check(got, q, codes, scales, n_vis, n, 0.04, where, group=group, which=some)
        again = run(fx, q, codes, scales, n_vis, n, 0.04, where, group=group, ws=ws)
        assert np.array_equal(got[0], again[0]) and np.array_equal(got[1], again[1])
        # the parts' borders lie elsewhere, and every run's results within the bounds of both
        whole = run(fx, q, codes, scales, n_vis, n, 0.04, where, group=group,
                    ws=torch.full((16,), 255, dtype=torch.uint8, device="cuda"))
        assert np.abs(got[0] - whole[0]).max() <= 2.0 ** -8 * max(np.abs(whole[0]).max(), 1.0)
        assert np.array_equal(np.isneginf(got[1]), np.isneginf(whole[1]))


def test_what_lies_behind_masks(fx):
    """rows that no query sees, and rows that only some queries of a block see, may hold NaN codes"""
    rng = np.random.default_rng(0)
    n, group, heads, window = 150, 6, 7, 40
    codes, scales = cache(rng, n)
    n_vis = np.array([60, 61, 62, 0, 130, 131], np.int32)
    q = bf16(rng.standard_normal((group, heads, 512)))
    where = dict(kv_base=np.zeros(1, np.int64))
    want = run(fx, q, codes, scales, n_vis, n, 0.05, where, window=window, group=group)
    check(want, q, codes, scales, n_vis, n, 0.05, where, window=window, group=group)
    unseen = np.r_[0:20, 62:90, 131:150]
    codes[unseen], scales[unseen] = 0xFF, 0xFF
    got = run(fx, q, codes, scales, n_vis, n, 0.05, where, window=window, group=group)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    codes[61, 5] = 0x7F  # the entry that query 2 alone sees
    codes[20, 300] = 0xFF  # and query 0 alone
    got = run(fx, q, codes, scales, n_vis, n, 0.05, where, window=window, group=group)
    for t in range(group):
        if t in (0, 2):
            assert np.isnan(got[1][t]).all() and np.isnan(got[0][t]).all()
        else:
            assert np.array_equal(got[0][t], want[0][t]) and np.array_equal(got[1][t], want[1][t])


def test_queries_that_are_not_finite(fx):
    rng = np.random.default_rng(1)
    codes, scales = cache(rng, 100)
    q = bf16(rng.standard_normal((4, 9, 512)))
    where, n_vis = dict(kv_base=np.zeros(2, np.int64)), np.array([70, 71, 90, 0], np.int32)
    want = run(fx, q, codes, scales, n_vis, 100, 0.05, where, window=64, group=2)
    q[0, 2, 100], q[1, 8, 0], q[2, 0, 511], q[3, 1, 1] = np.nan, np.inf, -np.inf, np.nan
    got = run(fx, q, codes, scales, n_vis, 100, 0.05, where, window=64, group=2)
    bad = np.zeros((4, 9), bool)
    bad[0, 2] = bad[1, 8] = bad[2, 0] = True
    assert np.isnan(got[1][bad]).all() and np.isnan(got[0][bad]).all()
    assert np.array_equal(got[0][~bad], want[0][~bad]) and np.array_equal(got[1][~bad], want[1][~bad])


def test_entries_that_are_not_there(fx):
    rng = np.random.default_rng(2)
    where, rows = where_of("odd", rng, 4, 100, 0)
    codes, scales = cache(rng, rows)
    where["pages"][where["seq"][0], 12] = -1
    where["pages"][where["seq"][0], 13] = rows // 7
    where["seq"][1], where["seq"][2] = -1, 6
    n_vis = np.full(8, 95, np.int32)
    q = bf16(rng.standard_normal((8, 20, 512)))
    for window in (0, 30):
        got = run(fx, q, codes, scales, n_vis, 100, 0.05, where, window=window, group=2)
        check(got, q, codes, scales, n_vis, 100, 0.05, where, window=window, group=2)
        assert np.isneginf(got[1][2:6]).all() and (got[0][2:6] == 0).all()
    none = run(fx, q, codes[:0], scales[:0], n_vis, 100, 0.05, where, group=2)
    assert np.isneginf(none[1]).all() and (none[0] == 0).all()
    base = dict(kv_base=np.array([-50, rows - 40, -(1 << 62), 1 << 62], np.int64))
    got = run(fx, q, codes, scales, n_vis, 100, 0.05, base, group=2)
    check(got, q, codes, scales, n_vis, 100, 0.05, base, group=2)


def test_extreme_values_and_logits(fx):
    """the format's largest and smallest values, logits that rise all along and lie far apart"""
    rng = np.random.default_rng(3)
    n = 400
    y = rng.standard_normal((n, 512))
    y[:100] *= 2.0 ** -18
    y[100:200] *= 2.0 ** 14
    codes, scales = rows_ref.quantise("local", y)
    where, n_vis = dict(kv_base=np.zeros(1, np.int64)), np.array([n, n - 1], np.int32)
    q = bf16(rng.standard_normal((2, 16, 512)))
    for scale in (2.0 ** -20, 0.001, 0.0, -0.0005):
        got = run(fx, q, codes, scales, n_vis, n, scale, where, group=2)
        check(got, q, codes, scales, n_vis, n, scale, where, group=2)
    y = np.abs(y[200:201]) * np.linspace(0.01, 1.0, n)[:, None]
    codes, scales = rows_ref.quantise("local", y)
    q = np.abs(q)
    for scale in (0.5, -0.5):
        got = run(fx, q, codes, scales, n_vis, n, scale, where, group=2)
        check(got, q, codes, scales, n_vis, n, scale, where, group=2)


@pytest.mark.parametrize("nq, heads", [(5, 37), (240, 64)])
def test_one_query_of_few_entries(fx, nq, heads):
    """the single query's ways out: hidden rows and absent ones, queries that are not finite, logits far apart"""
    rng = np.random.default_rng(heads)
    n, few = 150, [0, 1, 2, 3, 4, nq - 1]
    codes, scales = cache(rng, 3 * n)
    codes[n:2 * n], scales[n:2 * n] = 0xFF, 0xFF  # of no sequence
    rises = np.abs(rng.standard_normal((1, 512))) * np.linspace(0.01, 1.0, n)[:, None]
    codes[2 * n:], scales[2 * n:] = rows_ref.quantise("local", rises)
    pages = np.array([[0, 1, 2], [6, 7, 8], [0, -1, 2], [6, 1, 9], [3, 4, 5]], np.int32)
    seq = rng.integers(0, 4, nq).astype(np.int32)
    seq[:5] = [0, 1, 2, 3, 7]
    n_vis = rng.integers(100, n + 1, nq).astype(np.int32)
    q = bf16(rng.standard_normal((nq, heads, 512)))
    q[:, 1] = np.abs(q[:, 1])
    where = dict(pages=pages, page_size=50, seq=seq)
    for scale in (0.05, -0.3, 1.0):
        got = run(fx, q, codes, scales, n_vis, n, scale, where, window=110)
        check(got, q, codes, scales, n_vis, n, scale, where, window=110, which=few)
    assert np.isneginf(got[1][4]).all() and (got[0][4] == 0).all()
    q[0, 2, 100], q[1, 0, 0], q[2, 5, 511], q[3, 36, 17], q[4, 1, 1] = np.nan, np.inf, -np.inf, np.nan, np.nan
    bad = np.zeros((nq, heads), bool)
    bad[0, 2] = bad[1, 0] = bad[2, 5] = bad[3, 36] = True
    again = run(fx, q, codes, scales, n_vis, n, 1.0, where, window=110)
    assert np.isnan(again[1][bad]).all() and np.isnan(again[0][bad]).all()
    assert np.array_equal(again[0][~bad], got[0][~bad]) and np.array_equal(again[1][~bad], got[1][~bad])
    # hidden by the window, by n_vis, and in the middle of what query 1 alone sees
    n_vis[:], seq[:], n_vis[1], seq[1] = 140, 0, 130, 1
    want = run(fx, q, codes, scales, n_vis, n, 0.05, where, window=100)
    codes[[3, 39, 140, 149]], scales[[0, 20, 145]], codes[2 * n + 60, 400] = 0xFF, 0xFF, 0xFF
    got = run(fx, q, codes, scales, n_vis, n, 0.05, where, window=100)
    assert np.isnan(got[1][1]).all() and np.isnan(got[0][1]).all()
    rest = np.arange(nq) != 1
    assert np.array_equal(got[0][rest], want[0][rest], equal_nan=True)
    assert np.array_equal(got[1][rest], want[1][rest], equal_nan=True)


def test_a_cache_past_32_bits(fx):
    rng = np.random.default_rng(4)
    rows = (1 << 23) + 300
    codes = torch.full((rows, 512), 255, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, 16), 255, dtype=torch.uint8, device="cuda")
    c, s = cache(rng, 200)
    first = rows - 210
    codes[first:first + 200], scales[first:first + 200] = dev(c), dev(s)
    q = dev(bf16(rng.standard_normal((2, 64, 512)))).bfloat16()
    ws = fx.workspace(fx.IDX_OP_ATTEND_LOCAL, 2, 200, 64)
    outs = []
    nv = torch.tensor([150, 200], dtype=torch.int32, device="cuda")
    table = torch.tensor([[(rows - 300) // 100 + 1, (rows - 300) // 100 + 2]], dtype=torch.int32, device="cuda")
    pages = torch.full((60, 2), -1, dtype=torch.int32, device="cuda")
    pages[41:43] = table
    small_c, small_s = dev(c), dev(s)
    for kw in (dict(codes=codes, scales=scales, kv_base=torch.full((2,), first, device="cuda")),
               dict(codes=small_c, scales=small_s, kv_base=torch.zeros(2, dtype=torch.int64, device="cuda"))):
        out, lse = torch.empty_like(q), torch.empty(2, 64, device="cuda")
        fx.idx_attend_local(q, kw["codes"], kw["scales"], nv, 200, 0.05, out, ws, lse=lse, kv_base=kw["kv_base"])
        outs.append((out, lse))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    page0 = int(table[0, 0]) * 100
    codes[page0:page0 + 200], scales[page0:page0 + 200] = small_c, small_s
    out, lse = torch.empty_like(q), torch.empty(2, 64, device="cuda")
    fx.idx_attend_local(q, codes, scales, nv, 200, 0.05, out, ws, lse=lse, pages=pages, page_size=100,
                        seq=torch.tensor([41, 42], dtype=torch.int32, device="cuda"))
    assert torch.equal(out, outs[1][0]) and torch.equal(lse, outs[1][1])


def test_the_last_entries_of_the_largest_ring(fx):
    rng = np.random.default_rng(5)
    where, rows = where_of("odd", rng, 2, 0, 133)
    codes, scales = cache(rng, rows)
    n_vis = np.array([(1 << 30) - 1, 1 << 30, (1 << 30) - 77, 133], np.int32)
    q = bf16(rng.standard_normal((4, 10, 512)))
    kw = dict(window=128, ring=133, group=2)
    got = run(fx, q, codes, scales, n_vis, 1 << 30, 0.05, where, **kw)
    check(got, q, codes, scales, n_vis, 1 << 30, 0.05, where, which=[0, 1, 2], **kw)


def test_a_long_run_of_one_head(fx):
    rng = np.random.default_rng(8)
    nq, n = 65535, 65700
    where = dict(pages=rng.integers(0, 200, (1, -(-n // 7))).astype(np.int32), page_size=7, seq=np.zeros(1, np.int32))
    codes, scales = cache(rng, 1400)
    q = bf16(2 * rng.standard_normal((nq, 1, 512), dtype=np.float32))
    n_vis = (n - nq + 1 + np.arange(nq)).astype(np.int32)
    kw = dict(window=100, group=nq)
    got = run(fx, q, codes, scales, n_vis, n, 0.05, where, **kw)
    check(got, q, codes, scales, n_vis, n, 0.05, where, which=[0, 1, nq - 2, nq - 1, *rng.choice(nq, 40, replace=False)], **kw)


@pytest.mark.parametrize("window", [3, 0])
def test_rows_past_32_bits(fx, window):
    """65535 queries of 128 heads: more than 2^32 values"""
    rng = np.random.default_rng(9)
    nq, heads, n = 65535, 128, 5
    codes, scales = cache(rng, 60)
    q = torch.empty(nq, heads, 512, dtype=torch.bfloat16, device="cuda").normal_()
    base = np.arange(nq, dtype=np.int64) % 56
    n_vis = np.full(nq, n, np.int32)
    out, lse = torch.zeros_like(q), torch.zeros(nq, heads, device="cuda")
    ws = fx.workspace(fx.IDX_OP_ATTEND_LOCAL, nq, n, heads)
    fx.idx_attend_local(q, dev(codes), dev(scales), dev(n_vis), n, 0.05, out, ws, lse=lse, window=window, kv_base=dev(base))
    for t in (0, 32767, 32768, nq - 1):
        few = (slice(t, t + 1),)
        check((out[few].double().cpu().numpy(), lse[few].double().cpu().numpy()), q[few].float().cpu().numpy(), codes, scales,
              n_vis[few], n, 0.05, dict(kv_base=base[few]), window=window)


def test_in_place_of_the_other_part(fx):
    rng = np.random.default_rng(6)
    where, rows = where_of("base", rng, 40, 140, 0)
    codes, scales = cache(rng, rows)
    q = bf16(rng.standard_normal((40, 64, 512)))
    n_vis, pos = np.full(40, 140, np.int32), np.arange(40) * 1000
    other, other_lse = bf16(rng.standard_normal((40, 64, 512))), np.float32(rng.standard_normal((40, 64)) + 2)
    turn = (FREQ, 448, "half", 1.25)
    for window in (128, 0):
        want = run(fx, q, codes, scales, n_vis, 140, 0.05, where, other=other, other_lse=other_lse, turn=turn, pos=pos,
                   window=window)
        out, lse = dev(other).bfloat16(), dev(other_lse)
        ws = fx.workspace(fx.IDX_OP_ATTEND_LOCAL, 40, 140, 64)
        fx.idx_attend_local(dev(q).bfloat16(), dev(codes), dev(scales), dev(n_vis), 140, 0.05, out, ws, lse=lse, other=out,
                            other_lse=lse, kv_base=dev(where["kv_base"]), pos=dev(pos), freq=dev(FREQ), offset=448,
                            layout="half", mscale=1.25, window=window)
        assert np.array_equal(out.double().cpu().numpy(), want[0]) and np.array_equal(lse.double().cpu().numpy(), want[1])


def test_two_graphs_with_one_workspace(fx):
    """captured on a side stream, replayed in turn with eager calls of other sizes between, each against its eager result"""
    g = torch.Generator(device="cuda").manual_seed(7)
    codes = torch.randint(0, 127, (5000, 512), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.full((5000, 16), 119, dtype=torch.uint8, device="cuda")
    ws = fx.workspace(fx.IDX_OP_ATTEND_LOCAL, 2, 5000, 64)
    assert ws.numel() > 16
    sizes = [(2, 64, 0), (1, 16, 0), (2, 64, 128)]
    state = []
    for nq, heads, window in sizes:
        q = torch.randn(nq, heads, 512, device="cuda", generator=g).bfloat16()
        state.append((q, torch.empty_like(q), torch.empty(nq, heads, device="cuda"),
                      torch.full((nq,), 5000, dtype=torch.int32, device="cuda"), torch.zeros(nq, dtype=torch.int64, device="cuda"), window))

    def call(s, out=None, lse=None):
        q, o, l, nv, base, window = s
        fx.idx_attend_local(q, codes, scales, nv, 5000, 0.02, o if out is None else out, ws, lse=l if lse is None else lse,
                            kv_base=base, window=window)

    graphs, side = [], torch.cuda.Stream()
    for s in state:
        call(s)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call(s)
        graphs.append(graph)
    for i in range(4):
        for s, graph in zip(state, graphs):
            s[0].normal_(generator=g)
            s[3].fill_(5000 - 37 * i)
            out, lse = torch.empty_like(s[1]), torch.empty_like(s[2])
            s[1].fill_(7), s[2].fill_(7)
            graph.replay()
            call(s, out, lse)
            torch.cuda.synchronize()
            assert torch.equal(out, s[1]) and torch.equal(lse, s[2])


def test_a_graph_whose_lengths_change(fx):
    """blocks shared out anew at each replay, other calls on the same workspace between"""
    g = torch.Generator(device="cuda").manual_seed(11)
    n, runs, group, heads = 16384, 16, 2, 64
    codes = torch.randint(0, 127, (n, 512), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.full((n, 16), 119, dtype=torch.uint8, device="cuda")
    q = torch.randn(runs * group, heads, 512, device="cuda", generator=g).bfloat16()
    n_vis = torch.full((runs * group,), n, dtype=torch.int32, device="cuda")
    base = torch.zeros(runs, dtype=torch.int64, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(runs * group, heads, device="cuda")
    ws = fx.workspace(fx.IDX_OP_ATTEND_LOCAL, runs * group, n, heads)

    def call(out, lse, ws):
        fx.idx_attend_local(q, codes, scales, n_vis, n, 0.02, out, ws, lse=lse, group=group, kv_base=base)

    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        call(out, lse, ws)
    want, want_lse, own = torch.empty_like(q), torch.empty_like(lse), torch.full_like(ws, 255)
    one = torch.empty_like(q[:2]), torch.empty(2, heads, device="cuda")
    for _ in range(5):
        last = torch.randint(-1, n + 1, (runs, 1), device="cuda", generator=g)
        n_vis.copy_((last + torch.arange(group, device="cuda")).reshape(-1))
        q.normal_(generator=g)
        graph.replay()
        fx.idx_attend_local(q[:2], codes, scales, n_vis[:2], n, 0.02, one[0], ws, lse=one[1], group=2, kv_base=base[:1])
        call(want, want_lse, own)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
        own.fill_(255)
