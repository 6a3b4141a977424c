"""Distillation of score rows from a teacher's top logits (idx_distill, idx_distill_bwd) against the
definition in 64 bits."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fx():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import top_fp4_lightning_amd

    return top_fp4_lightning_amd


def reference(scores, n_vis, max_n, t_idx, t_logit, inv_temp, dloss):
    """per row: (loss, gradient over the visible positions, lse, t_lse) in 64 bits"""
    res = []
    for t in range(len(n_vis)):
        n = min(max(int(n_vis[t]), 0), max_n)
        s = scores[t, :n].astype(np.float64) * inv_temp
        keep = [i for i, p in enumerate(t_idx[t]) if 0 <= p < n and s[p] > -np.inf and t_logit[t, i] > -np.inf]
        with np.errstate(divide="ignore", invalid="ignore"):
            m = s.max(initial=-np.inf)
            lse = m + np.log(np.exp(s - (m if np.isfinite(m) else 0)).sum()) if np.isfinite(m) else -np.inf
        g = np.zeros(n)
        if not keep:
            res.append((0.0, g, lse, -np.inf))
            continue
        at = t_idx[t][keep]
        x = t_logit[t][keep].astype(np.float64) * inv_temp
        tl = x.max() + np.log(np.exp(x - x.max()).sum())
        p = np.exp(x - tl)
        loss = (p * ((x - tl) - (s[at] - lse))).sum()
        g = np.exp(s - lse)
        np.subtract.at(g, at, p)
        res.append((loss, g * float(dloss[t]) * inv_temp, lse, tl))
    return res


def check(fx, scores, n_vis, max_n, t_idx, t_logit, inv_temp=1.0, in_place=False):
    """tolerances: lse rounds to fp32 (2^-24 |lse|), its sum has n fp32 terms joined in a tree of at most 20 levels
    behind runs of at most n / 256 additions, each 2^-24, terms good to 2^-22 and |s| 2^-22; the loss is a sum in 64
    bits of terms p (log p - log q) with p good to 2^-22 (1 + |x|); the gradient's q and p are exponentials of
    differences good to 2^-22 (1 + |s| + |lse|)."""
    nq, k = t_idx.shape
    rng = np.random.default_rng(nq)
    dl = rng.standard_normal(nq).astype(np.float32)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    pad = np.full((nq, scores.shape[1] + 5), 3.0, np.float32)
    pad[:, :scores.shape[1]] = scores
    sd = dev(pad)[:, :max(scores.shape[1], 1)]
    nv, ti, tl = dev(np.asarray(n_vis, np.int32)), dev(t_idx.astype(np.int32)), dev(t_logit.astype(np.float32))
    loss, lse, tlse = (torch.full((nq,), 9.0, device="cuda") for _ in range(3))
    ws = fx.workspace(fx.IDX_OP_DISTILL, nq, max_n, 1)
    print(f"distill nq={nq} max_n={max_n} k={k} inv_temp={inv_temp}", flush=True)
    fx.idx_distill(sd, nv, max_n, ti, tl, loss, lse, tlse, ws, inv_temp=inv_temp)
    grad = sd if in_place else torch.full_like(sd, 7.0)
    before = grad.clone()
    fx.idx_distill_bwd(sd, nv, max_n, ti, tl, lse, tlse, dev(dl), grad, inv_temp=inv_temp)
    torch.cuda.synchronize()
    for t, (want, g, l, tl_) in enumerate(reference(scores, n_vis, max_n, t_idx, t_logit.astype(np.float32), inv_temp, dl)):
        n = len(g)
        fin = scores[t, :n][np.isfinite(scores[t, :n])]
        big = max(np.abs(fin).max(initial=0.0), np.abs(t_logit[t][np.isfinite(t_logit[t])]).max(initial=0.0)) * inv_temp
        e = 2.0 ** -22 * (2 + big) + n / 256 * 2.0 ** -24
        for got, ideal in ((lse, l), (tlse, tl_)):
            x = float(got[t])
            assert x == ideal if not np.isfinite(ideal) else abs(x - ideal) <= e + 2.0 ** -23 * abs(ideal), (t, x, ideal)
        with np.errstate(over="ignore"):  # scores near fp32's lowest: any loss is within its own rounding
            loss_tol = e * (2 + abs(want)) + 2.0 ** -24 * abs(want) + e * big
        assert abs(float(loss[t]) - want) <= loss_tol, (t, float(loss[t]), want)
        got = grad[t].double().cpu().numpy()
        at_p = np.zeros(n)
        live = (t_idx[t] >= 0) & (t_idx[t] < n)
        if np.isfinite(tl_):
            x = t_logit[t].astype(np.float64)[live] * inv_temp - tl_
            np.add.at(at_p, t_idx[t][live], np.exp(x))
        scale = abs(float(dl[t])) * inv_temp
        # q and p separately: their difference may cancel; p is of several slots at most k
        q = np.zeros(n) if not np.isfinite(l) else np.exp(scores[t, :n].astype(np.float64) * inv_temp - l)
        tol = (q + at_p) * scale * (4 * e + 2.0 ** -22 * abs(l if np.isfinite(l) else 0) + k * 2.0 ** -24)
        # exponentials and products below fp32's least normal number may come out as 0: 2^-126 each of q and p,
        # and of the product with the gain
        tol = tol + 2.0 ** -126 * (2 * scale + 1)
        assert (np.abs(got[:n] - g) <= tol).all(), (t, np.abs(got[:n] - g).max())
        assert (grad[t, n:] == before[t, n:]).all(), t
    return loss


def rows(rng, nq, n, k, spread=3.0):
    s = (rng.standard_normal((nq, n)) * spread).astype(np.float32)
    idx = np.stack([rng.permutation(n)[:k] if n >= k else np.r_[rng.permutation(n), [-1] * (k - n)] for _ in range(nq)])
    return s, idx, rng.standard_normal((nq, k)) * 2


@pytest.mark.parametrize("n", [1, 2, 3, 5, 63, 64, 255, 1000, 4095, 4096, 4097, 8200, 70001])
@pytest.mark.parametrize("k", [1, 7, 512])
def test_lengths(fx, n, k):
    rng = np.random.default_rng(n * 10 + k)
    s, idx, tl = rows(rng, 3, n, k)
    check(fx, s, [n, max(n - 3, 0), n // 2], n, idx, tl)


@pytest.mark.parametrize("nq,n,k", [(1, 300000, 2048), (1100, 77, 5), (1030, 4500, 64), (40, 9001, 300)])
def test_few_long_and_many_short_rows(fx, nq, n, k):
    rng = np.random.default_rng(nq)
    s, idx, tl = rows(rng, nq, n, k)
    check(fx, s, rng.integers(0, n + 1, nq), n, idx, tl)


@pytest.mark.parametrize("n,k", [(1, 1), (77, 5), (1023, 64), (1024, 100), (1025, 512), (2500, 300), (2500, 600)])
def test_many_short_rows(fx, n, k):
    rng = np.random.default_rng(n + k)
    nq = 2050
    s = (rng.standard_normal((nq, n)) * 3).astype(np.float32)
    s[rng.random((nq, n)) < 0.2] = -np.inf
    nv = rng.integers(0, n + 1, nq)
    nv[:3] = [n, 0, n]
    check(fx, s, nv, n, rng.integers(-1, n, (nq, k)), rng.standard_normal((nq, k)) * 2)


def test_a_gradient_beyond_the_last_level_cache(fx):
    """above 2^25 scores: most rows short, some of several pieces, the strides as wide as the longest"""
    rng = np.random.default_rng(9)
    nq, n, k = 1100, 31000, 40
    nv = rng.integers(0, 50, nq)
    nv[::150] = [n, n - 1, 4096, 8192, 8191, 12289, 20000, 30000]
    s = np.zeros((nq, n), np.float32)
    for t in range(nq):
        s[t, :nv[t]] = rng.standard_normal(nv[t]) * 3
    idx = (rng.random((nq, k)) * (nv[:, None] + 1)).astype(np.int64) - 1
    check(fx, s, nv, n, idx, rng.standard_normal((nq, k)) * 2)


@pytest.mark.parametrize("inv_temp", [0.25, 1.0, 3.0])
@pytest.mark.parametrize("spread", [0.1, 30.0])
def test_temperatures_and_spreads(fx, inv_temp, spread):
    rng = np.random.default_rng(3)
    s, idx, tl = rows(rng, 4, 5000, 100, spread)
    check(fx, s, [5000, 4999, 1234, 17], 5000, idx, tl, inv_temp)
    check(fx, s, [5000, 4999, 1234, 17], 5000, idx, tl, inv_temp, in_place=True)


def test_masked_scores_and_entries_left_out(fx):
    rng = np.random.default_rng(4)
    n, k = 6000, 90
    s, idx, tl = rows(rng, 8, n, k)
    s[0, rng.random(n) < 0.9] = -np.inf           # a pool
    s[1] = -np.inf                                # nothing to choose from
    s[2, idx[2]] = -np.inf                        # every entry masked
    idx[3] = -1                                   # no entry
    tl[4] = -np.inf                               # no logit
    tl[5, ::2] = -np.inf
    idx[5, 1::4] = 2 ** 31 - 1
    idx[6, :] = rng.integers(0, 20, k)            # positions given many times
    idx[7, 0], idx[7, 1] = -2 ** 31, n
    loss = check(fx, s, [n, n, n, n, n, n, n, 3], n, idx, tl)
    assert float(loss[1]) == float(loss[2]) == float(loss[3]) == float(loss[4]) == 0.0
    s[:, 4090:4100] = -3.0e38                     # the type's lowest values
    s[5, 7] = 3.0e38 / 4
    check(fx, s, [n, n, n, n, n, 7, n, 3], n, idx, tl)


def test_no_slots_and_no_positions(fx):
    rng = np.random.default_rng(5)
    s = rng.standard_normal((2, 10)).astype(np.float32)
    check(fx, s, [10, 0], 10, np.zeros((2, 0), int), np.zeros((2, 0)))
    check(fx, s[:, :0], [0, 0], 0, np.zeros((2, 3), int), np.zeros((2, 3)))


def test_a_position_given_often_sums_in_one_order(fx):
    rng = np.random.default_rng(8)
    n, k = 9000, 2048
    s, _, tl = rows(rng, 4, n, k)
    idx = rng.integers(0, n // 100, (4, k)) * 100
    check(fx, s, [n] * 4, n, idx, tl)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    args = (dev(s), dev(np.full(4, n, np.int32)), n, dev(idx.astype(np.int32)), dev(tl.astype(np.float32)))
    loss, lse, tlse, dl = (torch.ones(4, device="cuda") for _ in range(4))
    fx.idx_distill(*args, loss, lse, tlse, fx.workspace(fx.IDX_OP_DISTILL, 4, n, 1))
    g = [fx.idx_distill_bwd(*args, lse, tlse, dl, torch.empty(4, n, device="cuda")) for _ in range(20)]
    assert all(torch.equal(x, g[0]) for x in g)


def test_gradient_against_differences(fx):
    """central differences of the loss in 64 bits from the scores the call saw"""
    rng = np.random.default_rng(6)
    s, idx, tl = rows(rng, 1, 40, 9)
    inv = 0.5
    nv = torch.tensor([40], dtype=torch.int32, device="cuda")
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    loss, lse, tlse = (torch.empty(1, device="cuda") for _ in range(3))
    args = (dev(s), nv, 40, dev(idx.astype(np.int32)), dev(tl.astype(np.float32)))
    fx.idx_distill(*args, loss, lse, tlse, fx.workspace(fx.IDX_OP_DISTILL, 1, 40, 1), inv_temp=inv)
    g = torch.empty(1, 40, device="cuda")
    fx.idx_distill_bwd(*args, lse, tlse, torch.ones(1, device="cuda"), g, inv_temp=inv)
    f = lambda v: reference(v, [40], 40, idx, tl.astype(np.float32), inv, [1.0])[0][0]
    h = 1e-4
    for i in range(40):
        up, dn = s.astype(np.float64), s.astype(np.float64)
        up[0, i] += h
        dn[0, i] -= h
        # third differences: below h^2; the call: 2^-19
        assert abs((f(up) - f(dn)) / (2 * h) - float(g[0, i])) <= h * h + 2.0 ** -19


def test_replayed_graph_and_streams(fx):
    rng = np.random.default_rng(7)
    s, idx, tl = rows(rng, 5, 30000, 512)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    args = (dev(s), dev(np.full(5, 30000, np.int32)), 30000, dev(idx.astype(np.int32)), dev(tl.astype(np.float32)))
    ws = fx.workspace(fx.IDX_OP_DISTILL, 5, 30000, 1)
    loss, lse, tlse, dl = (torch.ones(5, device="cuda") for _ in range(4))
    g = torch.zeros(5, 30000, device="cuda")

    def step(stream=None):
        fx.idx_distill(*args, loss, lse, tlse, ws, inv_temp=0.7, stream=stream)
        fx.idx_distill_bwd(*args, lse, tlse, dl, g, inv_temp=0.7, stream=stream)

    step()
    torch.cuda.synchronize()
    want = loss.clone(), g.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for rep in range(3):
        loss.zero_()
        g.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(loss, want[0]) and torch.equal(g, want[1]), rep
    loss.zero_()
    g.zero_()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    step(side)
    torch.cuda.synchronize()
    assert torch.equal(loss, want[0]) and torch.equal(g, want[1])
