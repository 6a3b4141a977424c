"""Calls of idx_attend_local that its documentation allows, at the ends of its arguments' ranges."""
import numpy as np
import pytest

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
