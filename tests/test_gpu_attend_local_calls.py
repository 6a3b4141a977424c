"""Calls of idx_attend_local that its documentation allows, at the ends of its arguments' ranges."""
import numpy as np
import pytest
import torch

from test_gpu_attend_local import bf16, cache, check, fx, run, where_of  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window", [2 ** 63 - 1, 2 ** 63 - 63, 2 ** 62, 2 ** 31, 200])
def test_windows_wider_than_any_range(fx, window):
    """several queries a block, which see more entries than their windows could lie apart in"""
    rng = np.random.default_rng(0)
    runs, group, heads, n = 2, 3, 7, 200
    where, rows = where_of("pages", rng, runs, n, 0)
    codes, scales = cache(rng, rows)
    q = bf16(rng.standard_normal((runs * group, heads, 512)))
    n_vis = (n - group + 1 + np.tile(np.arange(group), runs)).astype(np.int32)
    kw = dict(window=window, group=group)
    got = run(fx, q, codes, scales, n_vis, n, 0.05, where, ws=_workspace(fx, q, n), **kw)
    check(got, q, codes, scales, n_vis, n, 0.05, where, **kw)


def _workspace(fx, q, entries):
    return fx.workspace(fx.IDX_OP_ATTEND_LOCAL, q.shape[0], entries, q.shape[1])


@pytest.mark.parametrize("nq, heads", [(3, 128), (300, 64), (1000, 48), (700, 5)])
def test_logarithms_in_place(fx, nq, heads):
    """lse written over other_lse, by blocks of one and of several times 16 heads"""
    g = torch.Generator(device="cuda").manual_seed(nq)
    codes = torch.randint(0, 127, (4000, 512), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.full((4000, 16), 119, dtype=torch.uint8, device="cuda")
    q, other = (torch.randn(nq, heads, 512, device="cuda", generator=g).bfloat16() for _ in range(2))
    n_vis = torch.randint(0, 129, (nq,), device="cuda", generator=g).int()
    base = torch.randint(0, 3800, (nq,), device="cuda", generator=g)
    ws = fx.workspace(fx.IDX_OP_ATTEND_LOCAL, nq, 128, heads)
    for _ in range(5):
        other_lse = 4 * torch.randn(nq, heads, device="cuda", generator=g)
        out, lse = torch.empty_like(q), torch.empty_like(other_lse)
        fx.idx_attend_local(q, codes, scales, n_vis, 128, 0.02, out, ws, lse=lse, other=other, other_lse=other_lse, kv_base=base)
        o2, l2 = other.clone(), other_lse.clone()
        fx.idx_attend_local(q, codes, scales, n_vis, 128, 0.02, o2, ws, lse=l2, other=o2, other_lse=l2, kv_base=base)
        assert torch.equal(out, o2) and torch.equal(lse, l2)
