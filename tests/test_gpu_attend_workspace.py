"""idx_attend in workspaces of other calls' sizes: shorter contexts, smaller batches and the least workspace, with
nothing written outside it."""
import numpy as np
import pytest
import torch

import attn_ref as ref

pytestmark = pytest.mark.gpu
SCALE = 512 ** -0.5


@pytest.fixture(scope="module")
def fx():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import top_fp4_lightning_amd

    return top_fp4_lightning_amd


def attend(fx, nq, heads, n, ws_bytes, long=()):
    """queries of a few entries, those of `long` of n; checked against the definition in 64 bits. The tolerance with
    the rows' own largest magnitude in place of the format's: the probabilities that round to zero are below 2^-31."""
    rng = np.random.default_rng(nq + n)
    rows = n + 40
    codes = rng.integers(0, 256, (rows, 256), dtype=np.uint8)
    scales = rng.integers(0x18, 0x2C, (rows, 32), dtype=np.uint8)
    n_vis = rng.integers(0, min(n, 70) + 1, nq)
    n_vis[list(long)] = n - np.arange(len(long)) % min(n, 40)
    base = rng.integers(0, 40, nq)
    q = torch.from_numpy(rng.standard_normal((nq, heads, 512)).astype(np.float32) * 2).bfloat16()
    dev = lambda a, dt: torch.from_numpy(np.ascontiguousarray(a, dtype=dt)).cuda()
    room = torch.full((ws_bytes + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    ws = room[256:256 + ws_bytes]
    out, lse = torch.empty(nq, heads, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(nq, heads, device="cuda")
    print(f"attend nq={nq} heads={heads} n={n} ws={ws_bytes}", flush=True)
    fx.idx_attend(q.cuda(), dev(codes, np.uint8), dev(scales, np.uint8), dev(n_vis, np.int32), n, SCALE, out, ws, lse=lse,
                  kv_base=dev(base, np.int64))
    torch.cuda.synchronize()
    assert (room[:256] == 0xA5).all() and (room[256 + ws_bytes:] == 0xA5).all()
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    most = np.abs(ref.kv_rows(codes, scales)).max()
    for t in set(long) | set(range(0, nq, max(1, nq // 16))):
        where = list(range(base[t], base[t] + n_vis[t]))
        r = ref.attention(q[t].double().numpy(), codes, scales, SCALE, where)
        m = max(len(where), 1)
        tol = ref.out_tolerance(r, m) - m * 2.0 ** -31 * (2688 - most)
        assert (np.abs(out[t] - r["out"]) <= tol).all(), (t, np.abs(out[t] - r["out"]).max())
        if where:
            assert (np.abs(lse[t] - r["lse"]) <= ref.lse_tolerance(r, m)).all(), t
        else:
            assert (out[t] == 0).all() and np.isneginf(lse[t]).all(), t


def test_the_size_of_a_longer_context(fx):
    """lengths whose own size is larger"""
    of = lambda n: fx.workspace_size(fx.IDX_OP_ATTEND, 100, n, 64)
    assert of(10560) > of(10624)
    attend(fx, 100, 64, 10560, of(10624), long=(0, 50, 99))
    attend(fx, 100, 64, 700, of(10624), long=(0, 1, 99))


@pytest.mark.parametrize("nq", [1, 2, 8, 15])
def test_the_size_of_a_larger_batch(fx, nq):
    size = fx.workspace_size(fx.IDX_OP_ATTEND, 16, 512, 64)
    assert fx.workspace_size(fx.IDX_OP_ATTEND, 8, 512, 64) > size
    attend(fx, nq, 64, 512, size, long=range(nq))


@pytest.mark.parametrize("heads", [1, 20, 64, 128])
@pytest.mark.parametrize("units", [0, 1, 2, 3, 5, 9])
def test_any_size(fx, heads, units):
    """one long query in room for any number of parts (sums and output of a head: 514 fp32), and a little less"""
    each = heads * 514 * 4
    for ws_bytes in {max(units * each, 16), max((units + 1) * each - 16, 16)}:
        attend(fx, 1, heads, 9000, ws_bytes, long=(0,))
        attend(fx, 3, heads, 3000, ws_bytes, long=(0, 2))


def test_less_than_the_least_is_refused(fx):
    for ws_bytes in (0, 8, 15):
        with pytest.raises(fx.IdxError) as e:
            attend(fx, 1, 4, 64, ws_bytes, long=(0,))
        assert e.value.status == fx.IDX_EWORKSPACE
