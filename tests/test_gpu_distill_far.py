"""Distillation of rows whose scores or logits lie far from zero, down to the type's lowest value everywhere (a mask
that is not -inf and leaves nothing): only differences count. Against the definition in 64 bits, shifted first."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
LOWEST = np.finfo(np.float32).min


@pytest.fixture(scope="module")
def fx():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import top_fp4_lightning_amd

    return top_fp4_lightning_amd


def check(fx, scores, n_vis, t_idx, t_logit, inv_temp, in_place=False):
    """Tolerances, relative to q, p and the terms of the loss. A difference to the largest is rounded once and
    multiplied by a factor of three roundings: 2^-22 |d| with d = (x - largest) / T; its exponential 2^-22; the sum of
    n terms, 2^-24 for each of the n / 256 + 24 additions behind one another, and the terms' own errors again, which
    are below 2^-22 as exp(-|d|) |d| < 1. Where both logarithms lie within 1024 the gradient takes them as stored:
    half a step of fp32, 2^-24 of each. Values below 2^-125 may be zero."""
    nq, n = scores.shape
    k = t_idx.shape[1]
    dev = lambda a, dt: torch.from_numpy(np.ascontiguousarray(a, dtype=dt)).cuda()
    s, nv, ti, tl = dev(scores, np.float32), dev(n_vis, np.int32), dev(t_idx, np.int32), dev(t_logit, np.float32)
    dl = np.linspace(0.5, 2.0, nq).astype(np.float32)
    loss, lse, tlse = (torch.full((nq,), 9.0, device="cuda") for _ in range(3))
    print(f"distill far nq={nq} n={n} k={k} inv_temp={inv_temp} in_place={in_place}", flush=True)
    fx.idx_distill(s, nv, n, ti, tl, loss, lse, tlse, fx.workspace(fx.IDX_OP_DISTILL, nq, n, 1), inv_temp=inv_temp)
    grad = s if in_place else torch.full_like(s, 7.0)
    fx.idx_distill_bwd(s, nv, n, ti, tl, lse, tlse, dev(dl, np.float32), grad, inv_temp=inv_temp)
    torch.cuda.synchronize()
    grad, loss = grad.double().cpu().numpy(), loss.double().cpu().numpy()
    for t in range(nq):
        x = scores[t, :n_vis[t]].astype(np.float64)
        keep = [i for i in range(k) if 0 <= t_idx[t, i] < n_vis[t] and x[t_idx[t, i]] > -np.inf and t_logit[t, i] > -np.inf]
        if not keep:
            assert loss[t] == 0.0 and (grad[t, :n_vis[t]] == 0.0).all(), t
            continue
        at = t_idx[t, keep]
        ds, y = (x - x.max()) * inv_temp, t_logit[t, keep].astype(np.float64)
        dt = (y - y.max()) * inv_temp
        ls, lt = np.log(np.exp(ds).sum()), np.log(np.exp(dt).sum())
        p = np.exp(dt - lt)
        term = (dt - lt) - (ds[at] - ls)
        rel = lambda d: 2.0 ** -21 * (2 + np.where(np.isfinite(d), np.abs(d), 0)) + (n / 256 + 24) * 2.0 ** -24
        logs = abs(x.max() * inv_temp + ls), abs(y.max() * inv_temp + lt)
        near = 2.0 ** -24 * 1.01 * max(logs) if max(logs) < 1025 else 0.0
        want = (p * term).sum()
        # p is an exponential in fp32; the two logarithms have the sums' errors
        tol = (p * np.abs(term) * rel(dt)).sum() + 2 * rel(0.0) + 2.0 ** -24 * abs(want)
        assert abs(loss[t] - want) <= tol, (t, loss[t], want, tol)
        q = np.exp(ds - ls)
        g, size = q.copy(), q * (rel(ds) + near)
        np.subtract.at(g, at, p)
        np.add.at(size, at, p * (rel(dt) + near + k * 2.0 ** -24))
        gain = float(dl[t]) * inv_temp
        tol = size * gain * 1.01 + 2.0 ** -22 * np.abs(g) * gain + 2.0 ** -125 * (1 + gain)
        err = np.abs(grad[t, :n_vis[t]] - g * gain)
        assert (err <= tol).all(), (t, err.max(), tol[err.argmax()])


def teacher(rng, nq, n, k):
    return np.stack([rng.permutation(n)[:k] for _ in range(nq)]), (rng.standard_normal((nq, k)) * 2).astype(np.float32)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("nq,n,k", [(3, 1, 1), (3, 77, 9), (2, 5000, 300), (2, 70001, 512), (1100, 5000, 40), (2050, 900, 33)])
def test_rows_of_the_lowest_value(fx, nq, n, k, in_place):
    """every position at the lowest value but those that are -inf: equal probabilities; some rows ordinary"""
    rng = np.random.default_rng(n)
    idx, tl = teacher(rng, nq, n, k)
    s = np.full((nq, n), LOWEST, np.float32)
    s[1::5] = rng.standard_normal(s[1::5].shape)
    s[2::5, ::3] = -np.inf
    tl[0] = LOWEST
    check(fx, s, [n - (t % 3) * (n // 4) for t in range(nq)], idx, tl, 1.0, in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("shift,inv_temp", [(500.0, 1.0), (-900.0, 1.0), (3000.0, 0.5), (-1.0e6, 2.0), (2.0 ** 30, 1.0)])
def test_rows_far_from_zero(fx, shift, inv_temp, in_place):
    """rows shifted by more than their spread: the scores, the logits or both (rounded as inputs)"""
    rng = np.random.default_rng(5)
    nq, n, k = 6, 9000, 200
    idx, tl = teacher(rng, nq, n, k)
    s = (rng.standard_normal((nq, n)) * 3).astype(np.float32)
    s[0::3] += np.float32(shift)
    tl[1::3] -= np.float32(shift)
    s[2::3] -= np.float32(shift)
    tl[2::3] += np.float32(shift)
    n_vis = [n, n - 1, 4096, 4097, 8192, 300]
    check(fx, s, n_vis, idx, tl, inv_temp, in_place)
    check(fx, np.where(rng.random(s.shape) < 0.9, np.float32(-np.inf), s), n_vis, idx, tl, inv_temp, in_place)
