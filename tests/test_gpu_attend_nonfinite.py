"""A query row that is not finite: its head is NaN, whatever sign its products have, and no other head is touched."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fx():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import top_fp4_lightning_amd

    return top_fp4_lightning_amd


def cache(rows):
    """value 0 of every row is -1, value 1 is +2, value 2 is 0, the others are mixed"""
    rng = np.random.default_rng(1)
    codes = rng.integers(0, 256, (rows, 256), dtype=np.uint8)
    codes[:, 0] = 0xA | (4 << 4)
    codes[:, 1] = (codes[:, 1] & 0xF0)
    scales = np.full((rows, 32), 0x38, np.uint8)
    return torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()


@pytest.mark.parametrize("scale", [0.05, -0.05])
@pytest.mark.parametrize("at,value", [(0, np.inf), (0, -np.inf), (1, np.inf), (1, -np.inf), (2, np.inf), (5, -np.inf), (7, np.nan)])
@pytest.mark.parametrize("n,heads", [(1, 1), (1, 64), (3, 20), (64, 40), (130, 64), (20000, 3)])
def test_the_head_is_nan(fx, n, heads, at, value, scale):
    """one entry (all products of one sign), a tile, several, parts that are joined; with a list whose other slots are
    empty; a query without entries stays zero"""
    codes, scales = cache(n)
    q = torch.randn(3, heads, 512, generator=torch.Generator().manual_seed(2)).bfloat16()
    bad = q.clone()
    h = heads // 2
    bad[0, h, at] = bad[2, h, at] = value
    nv = torch.tensor([n, n, 0], dtype=torch.int32, device="cuda")
    base = torch.zeros(3, dtype=torch.int64, device="cuda")
    idx = torch.full((3, 70), -1, dtype=torch.int32)
    idx[:, 66] = n - 1
    print(f"attend nonfinite n={n} heads={heads} at={at} value={value}", flush=True)
    for lst in (None, idx.cuda()):
        k = n if lst is None else 70
        res = []
        for x in (q.cuda(), bad.cuda()):
            out, lse = torch.empty_like(x), torch.empty(3, heads, device="cuda")
            fx.idx_attend(x, codes, scales, nv, n, scale, out, fx.workspace(fx.IDX_OP_ATTEND, 3, k, heads), lse=lse,
                          kv_base=base, idx=lst)
            w = torch.zeros(3, k, device="cuda")
            fx.idx_attend_weights(x, codes, scales, nv, n, scale, lse, w, kv_base=base, idx=lst)
            res.append((out.cpu(), lse.cpu(), w.cpu()))
        (o0, l0, w0), (o1, l1, w1) = res
        hit = torch.zeros(3, heads, dtype=torch.bool)
        hit[0, h] = True
        assert o1[hit].isnan().all() and l1[hit].isnan().all()
        assert torch.equal(o1[~hit], o0[~hit]) and torch.equal(l1[~hit], l0[~hit])
        assert (o1[2] == 0).all() and l1[2].isneginf().all()
        seen = slice(0, n) if lst is None else slice(66, 67)
        assert w1[0, seen].isnan().all() and torch.equal(w1[1:], w0[1:])
        if lst is not None:
            assert (w1[0, :66] == 0).all() and (w1[0, 67:] == 0).all()
