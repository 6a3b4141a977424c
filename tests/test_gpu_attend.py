"""Attention over the main-KV cache and its weights per position (idx_attend, idx_attend_weights)
against the definition in 64 bits."""
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


def cache(rng, rows):
    """codes of every value, scales of the usual size with a few subnormal, zero and negative ones"""
    codes = rng.integers(0, 256, (rows, 256), dtype=np.uint8)
    scales = rng.integers(0x18, 0x2C, (rows, 32), dtype=np.uint8)
    scales[::5, ::7] = rng.integers(0, 8, scales[::5, ::7].shape)
    scales[::11, 3] |= 0x80
    return codes, scales


def bf16(a):
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).bfloat16()
    return t.cuda(), t.double().numpy()


def dev(a, dt=None):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a if dt is None else np.asarray(a, dt))).cuda()


def check(fx, q, codes, scales, n_vis, max_n, scale=SCALE, kv_base=None, pages=None, page_size=0, seq=None, idx=None,
          window=0, weights=True, lse_given=None):
    """both calls against the definition, every query"""
    nq, heads = q.shape[:2]
    qd, q64 = bf16(q)
    cd, sd = dev(codes), dev(scales)
    where = dict(kv_base=dev(kv_base, np.int64), pages=dev(pages, np.int32), page_size=page_size,
                 seq=dev(seq, np.int32), idx=dev(idx, np.int32))
    nv = dev(n_vis, np.int32)
    entries = idx.shape[1] if idx is not None else (min(window, max_n) if window else max_n)
    ws = fx.workspace(fx.IDX_OP_ATTEND, nq, entries, heads)
    out = torch.full((nq, heads, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((nq, heads), 7.0, device="cuda")
    print(f"attend nq={nq} heads={heads} max_n={max_n} entries={entries} page={page_size} window={window}", flush=True)
    fx.idx_attend(qd, cd, sd, nv, max_n, scale, out, ws, lse=lse, window=window, **where)
    width = idx.shape[1] if idx is not None else max_n
    w = None
    if weights and not window:
        w = torch.full((nq, max(width, 1) + 3), 7.0, device="cuda")
        fx.idx_attend_weights(qd, cd, sd, nv, max_n, scale, lse, w, **where)
    torch.cuda.synchronize()
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for t in range(nq):
        slots, rows = ref.entries(t, n_vis, max_n, len(codes), kv_base, pages, page_size, seq, idx, window)
        r = ref.attention(q64[t], codes, scales, scale, rows)
        n = max(len(rows), 1)
        err = np.abs(out[t] - r["out"])
        assert (err <= ref.out_tolerance(r, n)).all(), (t, err.max(), np.abs(r["out"]).max())
        if not rows:
            assert (out[t] == 0).all() and np.isneginf(lse[t]).all(), t
        else:
            assert (np.abs(lse[t] - r["lse"]) <= ref.lse_tolerance(r, n)).all(), (t, np.abs(lse[t] - r["lse"]).max())
        if w is not None:
            got = w[t].double().cpu().numpy()
            want = np.full(w.shape[1], 7.0)
            if idx is not None:
                want[:width] = 0.0
            tol = np.zeros(w.shape[1])
            if rows:
                # from the lse that the call was given
                x = np.exp(r["s"] - lse[t][:, None]).mean(0)
                want[slots] = x
                tol[slots] = ref.weight_tolerance(r, x)
            elif idx is None:
                n_t = min(max(int(n_vis[t]), 0), max_n)
                want[:n_t] = 0.0  # visible, but no row of the cache
            if idx is None:  # visible positions without a row
                n_t = min(max(int(n_vis[t]), 0), max_n)
                hole = np.setdiff1d(np.arange(n_t), slots)
                want[hole] = 0.0
            assert (np.abs(got - want) <= tol).all(), (t, np.abs(got - want).max())
    return out, lse


@pytest.mark.parametrize("heads", [1, 5, 16, 31, 32, 33, 64, 100, 128])
def test_heads(fx, heads):
    rng = np.random.default_rng(heads)
    codes, scales = cache(rng, 400)
    idx = np.stack([rng.permutation(150)[:70] for _ in range(3)])
    check(fx, rng.standard_normal((3, heads, 512)) * 2, codes, scales, [150, 150, 149], 150, kv_base=[0, 100, 250],
          idx=idx)


@pytest.mark.parametrize("k", [1, 2, 15, 16, 17, 63, 64, 65, 128, 129, 512, 2048])
def test_list_lengths(fx, k):
    rng = np.random.default_rng(100 + k)
    n = 2500
    codes, scales = cache(rng, 2 * n)
    idx = np.stack([np.sort(rng.permutation(n)[:k]) for _ in range(2)])
    check(fx, rng.standard_normal((2, 64, 512)) * 2, codes, scales, [n, n - 7], n, kv_base=[0, n], idx=idx)


@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 127, 200, 1000])
@pytest.mark.parametrize("new", [1, 4])
def test_visible_range_of_a_chunk(fx, n, new):
    """causal: the i-th new token sees its own position and everything before"""
    new = min(new, n)
    rng = np.random.default_rng(200 + n)
    codes, scales = cache(rng, 2 * n)
    n_vis = [n - new + 1 + i for i in range(new)] * 2
    check(fx, rng.standard_normal((2 * new, 17, 512)) * 2, codes, scales, n_vis, n, kv_base=[0] * new + [n] * new)


@pytest.mark.parametrize("page", [1, 7, 16, 24, 64, 100, 256])
def test_pages(fx, page):
    """pages in any order that end inside a tile, sequences of different lengths, and a page that two share"""
    rng = np.random.default_rng(300 + page)
    per = -(-300 // page)
    codes, scales = cache(rng, (3 * per + 2) * page)
    pages = rng.permutation(3 * per + 2)[:3 * per].reshape(3, per)
    pages[1, 0] = pages[0, 0]
    seq = [0, 0, 1, 2, 2]
    n_vis = [299, 300, 131, 1, 65]
    q = rng.standard_normal((5, 40, 512)) * 2
    check(fx, q, codes, scales, n_vis, 300, pages=pages, page_size=page, seq=seq)
    idx = np.stack([rng.permutation(300)[:90] for _ in range(5)])
    check(fx, q, codes, scales, n_vis, 300, pages=pages, page_size=page, seq=seq, idx=idx)
    check(fx, q[:3], codes, scales, n_vis[:3], 300, pages=pages, page_size=page)  # query t is of sequence t


@pytest.mark.parametrize("window", [1, 3, 64, 100, 128, 500])
def test_window(fx, window):
    rng = np.random.default_rng(400 + window)
    codes, scales = cache(rng, 400)
    check(fx, rng.standard_normal((5, 20, 512)) * 2, codes, scales, [400, 399, 64, 1, 0], 400, kv_base=[0] * 5,
          window=window)


def test_rows_that_are_left_out(fx):
    """-1 padding, positions past the visible range, bad pages, sequences and bases, lists that leave nothing; what
    the cache holds at such rows (scales that are no numbers) has no effect"""
    rng = np.random.default_rng(5)
    codes, scales = cache(rng, 640)
    idx = np.full((6, 80), -1)
    idx[0, :5] = [3, 700, -9, 63, 2]
    idx[1] = rng.integers(100, 200, 80)      # all past the range
    idx[3, 79] = 0                           # one entry in the last slot
    idx[4, :40] = np.arange(40)
    idx[4, 20] = 2 ** 31 - 1
    idx[5] = -2 ** 31
    n_vis = [64, 100, 0, 64, 64, 64]
    q = rng.standard_normal((6, 64, 512)) * 2
    seen = set()
    for t in range(6):
        seen |= set(ref.entries(t, n_vis, 64, 640, kv_base=[64 * t] * 6, idx=idx)[1])
    poison = np.array(sorted(set(range(640)) - seen))
    scales[poison] = 0x7F
    check(fx, q, codes, scales, n_vis, 64, kv_base=[64 * t for t in range(6)], idx=idx)
    # a negative page, a page past the cache, sequence numbers outside, with and without a list
    scales[:] = rng.integers(0x18, 0x2C, scales.shape)
    pages = np.arange(40).reshape(4, 10)
    pages[0, 1], pages[1, 0], pages[2, 3] = -1, 40, 2 ** 31 - 1
    for lst in (None, np.stack([rng.permutation(160)[:50] for _ in range(6)])):
        check(fx, q, codes, scales, [160, 150, 159, 160, 160, 160], 160, pages=pages, page_size=16,
              seq=[0, 1, 2, 3, -1, 4], idx=lst)
        # a base that leaves part of the range, or all of it, outside the cache
        check(fx, q, codes, scales, [160] * 6, 160, kv_base=[-100, -160, 639, 640, 2 ** 62, -2 ** 62], idx=lst)
    # negative and too large n_vis are clamped
    check(fx, q[:2], codes, scales, [-5, 2 ** 31 - 1], 33, kv_base=[0, 0])


def test_an_empty_cache_and_empty_lists(fx):
    rng = np.random.default_rng(6)
    q = rng.standard_normal((2, 3, 512))
    none = np.zeros((0, 256), np.uint8), np.zeros((0, 32), np.uint8)
    check(fx, q, *none, [5, 0], 5, kv_base=[0, 0], idx=np.zeros((2, 4)))
    check(fx, q, *none, [5, 0], 5, kv_base=[0, 0])
    check(fx, q, *cache(rng, 8), [8, 8], 8, kv_base=[0, 0], idx=np.zeros((2, 0)))
    check(fx, q, *cache(rng, 8), [0, 0], 0, kv_base=[0, 0])


def test_a_position_listed_twice_counts_twice(fx):
    rng = np.random.default_rng(7)
    codes, scales = cache(rng, 100)
    idx = np.array([[5, 5, 5, 9, 9, 11, 5] + [50] * 93])
    check(fx, rng.standard_normal((1, 64, 512)) * 2, codes, scales, [100], 100, kv_base=[0], idx=idx)


@pytest.mark.parametrize("order", ["up", "down", "spike"])
@pytest.mark.parametrize("sharp", [8.0, 60.0])
def test_running_maximum(fx, order, sharp):
    """logits that grow, fall or jump along the entries: hundreds of units apart, so that early sums vanish"""
    rng = np.random.default_rng(8)
    n = 700
    codes, scales = cache(rng, n)
    q = rng.standard_normal((2, 64, 512))
    s = ref.kv_rows(codes, scales) @ q[0, 0]
    by = np.argsort(s)
    if order == "down":
        by = by[::-1]
    if order == "spike":
        by = np.roll(by[::-1], 333)
    check(fx, q * sharp, codes[by], scales[by], [n, n], n, kv_base=[0, 0])
    check(fx, q * sharp, codes, scales, [n, n], n, kv_base=[0, 0], idx=np.stack([by, by[::-1]]))


@pytest.mark.parametrize("power", [-120, -60, -20, 20, 60, 100])
def test_query_magnitudes(fx, power):
    """rows of any size (a power of two is taken off them), values of many sizes in a row, and zero rows"""
    rng = np.random.default_rng(9)
    codes, scales = cache(rng, 130)
    q = rng.standard_normal((2, 6, 512)) * 2.0 ** rng.integers(-20, 1, (2, 6, 512))
    q[0, 2] = 0.0
    q[1, 3, 1:] = 0.0
    check(fx, q * 2.0 ** power, codes, scales, [130, 100], 130, scale=SCALE * 2.0 ** -power, kv_base=[0, 0])


def test_a_query_row_that_is_not_finite_spoils_no_other(fx):
    rng = np.random.default_rng(10)
    codes, scales = cache(rng, 200)
    q = rng.standard_normal((3, 40, 512)).astype(np.float32)
    clean, _ = bf16(q)
    q[1, 7, 100], q[1, 33, 5] = np.nan, np.inf
    bad, _ = bf16(q)
    nv, base = dev([200, 200, 200], np.int32), dev([0, 0, 0], np.int64)
    outs = []
    for x in (clean, bad):
        out = torch.empty_like(x)
        fx.idx_attend(x, dev(codes), dev(scales), nv, 200, SCALE, out, fx.workspace(fx.IDX_OP_ATTEND, 3, 200, 40),
                      kv_base=base)
        outs.append(out.float().cpu())
    hit = torch.zeros(3, 40, dtype=torch.bool)
    hit[1, 7] = hit[1, 33] = True
    assert torch.equal(outs[0][~hit], outs[1][~hit])
    assert outs[1][hit].isnan().all()


@pytest.mark.parametrize("scale", [0.0, -0.05, 1.0])
def test_scales(fx, scale):
    rng = np.random.default_rng(11)
    codes, scales = cache(rng, 100)
    check(fx, rng.standard_normal((1, 4, 512)) * 0.2, codes, scales, [100], 100, scale=scale, kv_base=[0])


def test_one_token_over_a_long_range(fx):
    """split into parts and joined"""
    rng = np.random.default_rng(12)
    codes, scales = cache(rng, 20011)
    check(fx, rng.standard_normal((2, 3, 512)) * 4, codes, scales, [20011, 19000], 20011, kv_base=[0, 500])


@pytest.mark.parametrize("nq,heads,n", [(300, 2, 1000), (300, 40, 4096), (200, 16, 9000), (300, 20, 6000), (90, 64, 12000),
                                        (600, 5, 3000), (700, 16, 2000)])
def test_queries_in_unequal_numbers_of_parts(fx, nq, heads, n):
    """sizes at which some queries are cut into one part more than others (one and two, two and three, five and six):
    a few of full length on both sides of the change, the others short or empty"""
    rng = np.random.default_rng(17)
    codes, scales = cache(rng, n + 50)
    nv = rng.integers(0, 90, nq)
    for t in (0, 1, nq // 4, nq // 3, nq // 2, nq - 2, nq - 1):
        nv[t] = rng.integers(n - 100, n + 1)
    nv[2] = 0
    q = rng.standard_normal((nq, heads, 512)) * 2
    base = rng.integers(0, 50, nq)
    check(fx, q, codes, scales, nv, n, kv_base=base)
    if n <= 1000:
        idx = rng.integers(-1, n, (nq, n))
        check(fx, q, codes, scales, nv, n, kv_base=base, idx=idx)


def test_a_cache_beyond_32_bit_offsets(fx):
    rng = np.random.default_rng(13)
    rows = (1 << 24) + 1000  # 4.3 GB of codes
    part = cache(rng, 1000)
    codes = torch.zeros(rows, 256, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(rows, 32, dtype=torch.uint8, device="cuda")
    codes[-1000:], scales[-1000:] = dev(part[0]), dev(part[1])
    q, q64 = bf16(rng.standard_normal((2, 8, 512)) * 2)
    nv = dev([900, 1000], np.int32)
    pages = dev(np.arange((1 << 24) // 8, rows // 8)[None].repeat(2, 0), np.int32)
    for where in (dict(kv_base=dev([1 << 24] * 2, np.int64)), dict(pages=pages, page_size=8)):
        out, lse = torch.empty_like(q), torch.empty(2, 8, device="cuda")
        fx.idx_attend(q, codes, scales, nv, 1000, SCALE, out, fx.workspace(fx.IDX_OP_ATTEND, 2, 1000, 8), lse=lse, **where)
        for t, n in enumerate((900, 1000)):
            r = ref.attention(q64[t], *part, SCALE, list(range(n)))
            assert (np.abs(out[t].double().cpu().numpy() - r["out"]) <= ref.out_tolerance(r, n)).all()


def test_results_do_not_depend_on_the_batch_stride_or_stream(fx):
    """bit for bit the same twice, on another stream, from a replayed graph, with a strided list, and with what
    lies behind the outputs left as it was"""
    rng = np.random.default_rng(14)
    codes, scales = (dev(x) for x in cache(rng, 3000))
    q, _ = bf16(rng.standard_normal((4, 64, 512)) * 2)
    nv, base = dev([3000, 2500, 0, 700], np.int32), dev([0, 0, 0, 0], np.int64)
    wide = dev(np.stack([rng.permutation(3000)[:600] for _ in range(4)]), np.int32)
    idx = wide[:, :512]
    buf = torch.full((5, 64, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(4, 64, device="cuda")
    ws = fx.workspace(fx.IDX_OP_ATTEND, 4, 512, 64)

    def run(stream=None, lst=idx):
        buf[:4].fill_(9.0)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        fx.idx_attend(q, codes, scales, nv, 3000, SCALE, buf[:4], ws, lse=lse, kv_base=base, idx=lst, stream=stream)
        torch.cuda.synchronize()
        return buf[:4].clone(), lse.clone()

    a = run()
    for b in (run(), run(lst=idx.contiguous()), run(stream=torch.cuda.Stream())):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert (buf[4] == 3.0).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fx.idx_attend(q, codes, scales, nv, 3000, SCALE, buf[:4], ws, lse=lse, kv_base=base, idx=idx)
    for rep in range(3):
        buf.fill_(3.0)
        lse.fill_(0.0)
        (torch.randn(100, 100, device="cuda") @ torch.randn(100, 100, device="cuda")).sum()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a[0], buf[:4]) and torch.equal(a[1], lse), rep
    # a query by itself: another split, the same value up to the roundings of the joined sums
    one = torch.empty(1, 64, 512, dtype=torch.bfloat16, device="cuda")
    fx.idx_attend(q[1:2], codes, scales, nv[1:2], 3000, SCALE, one, fx.workspace(fx.IDX_OP_ATTEND, 1, 512, 64),
                  kv_base=base[1:2], idx=idx[1:2])
    assert (one[0].float() - a[0][1].float()).abs().max() <= 2.0 ** -7 * a[0][1].float().abs().max()


def test_scales_at_an_even_address(fx):
    rng = np.random.default_rng(15)
    part = cache(rng, 700)
    codes = dev(part[0])
    room = torch.full((700 * 32 + 6,), 0x7F, dtype=torch.uint8, device="cuda")  # NaN scales around
    q, _ = bf16(rng.standard_normal((3, 40, 512)) * 2)
    nv, base = dev([700, 333, 64], np.int32), dev([0, 0, 0], np.int64)
    idx = dev(np.stack([rng.permutation(700)[:90] for _ in range(3)]), np.int32)
    ws = fx.workspace(fx.IDX_OP_ATTEND, 3, 700, 40)
    got = []
    for off in (0, 2, 4, 6):
        room.fill_(0x7F)
        scales = room[off:off + 700 * 32].view(700, 32)
        scales.copy_(dev(part[1]))
        for lst in (None, idx):
            out, lse = torch.empty_like(q), torch.empty(3, 40, device="cuda")
            fx.idx_attend(q, codes, scales, nv, 700, SCALE, out, ws, lse=lse, kv_base=base, idx=lst)
            w = torch.zeros(3, 700 if lst is None else 90, device="cuda")
            fx.idx_attend_weights(q, codes, scales, nv, 700, SCALE, lse, w, kv_base=base, idx=lst)
            got.append((out, lse, w))
    for i, x in enumerate(got):
        assert all(torch.equal(a, b) and not b.isnan().any() for a, b in zip(got[i % 2], x)), i


def test_two_calls_at_once(fx):
    """on two streams, with workspaces of their own, both in parts that are joined"""
    rng = np.random.default_rng(16)
    codes, scales = (dev(x) for x in cache(rng, 30000))
    q, _ = bf16(rng.standard_normal((2, 2, 64, 512)) * 2)
    nv, base = dev([30000, 29000], np.int32), dev([0, 0], np.int64)
    ws = [fx.workspace(fx.IDX_OP_ATTEND, 2, 30000, 64) for _ in range(2)]
    assert ws[0].numel() > 16
    want = [torch.empty_like(q[0]) for _ in range(2)]
    for i in range(2):
        fx.idx_attend(q[i], codes, scales, nv, 30000, SCALE, want[i], ws[i], kv_base=base)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    out = [[torch.empty_like(q[0]) for _ in range(20)] for _ in range(2)]
    torch.cuda.synchronize()
    for rep in range(20):
        for i in range(2):
            fx.idx_attend(q[i], codes, scales, nv, 30000, SCALE, out[i][rep], ws[i], kv_base=base, stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in out[i])
