"""Steps of LayerAttention as programs make them: on another stream than the current one, recorded and replayed, with
sequences that change between steps."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fx():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import top_fp4_lightning_amd as fx

    return fx


@pytest.fixture(scope="module")
def pl(fx):
    from top_fp4_lightning_amd import pipeline

    return pipeline


# the kernels of one query, of windows (two of them) and of whole ranges, these in one part, in parts and shared out
@pytest.mark.parametrize("runs, group, heads, n, window", [
    (5, 3, 32, 140, 100), (9, 40, 16, 300, 64), (6, 5, 7, 400, 200), (6, 2, 24, 120, 0), (3, 2, 64, 3000, 0),
    (33, 3, 20, 8192, 0)])
@pytest.mark.parametrize("stride", ["group", 1, 0])
def test_sequences_of_any_stride(fx, runs, group, heads, n, window, stride):
    g = torch.Generator(device="cuda").manual_seed(runs)
    seqs, page = 4, 60
    per = -(-n // page)
    rows = seqs * per * page
    codes = torch.randint(0, 127, (rows, 512), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.full((rows, 16), 119, dtype=torch.uint8, device="cuda")
    pages = torch.randperm(seqs * per, device="cuda", generator=g).int().view(seqs, per)
    q = torch.randn(runs * group, heads, 512, device="cuda", generator=g).bfloat16()
    n_vis = torch.full((runs * group,), n, dtype=torch.int32, device="cuda")
    seq = torch.randint(0, seqs, (runs,), device="cuda", generator=g).int()
    if stride == "group":
        wide = torch.randint(-1, seqs + 1, (runs, group), device="cuda", generator=g).int()
        wide[:, 0] = seq
        view = wide.view(-1)[::group]
    elif stride == 1:
        view = seq
    else:
        seq = seq[:1].expand(runs).contiguous()
        view = seq[:1].expand(runs)
    ws = fx.workspace(fx.IDX_OP_ATTEND_LOCAL, runs * group, n, heads)
    got = []
    for s in (seq, view):
        out, lse = torch.empty_like(q), torch.empty(runs * group, heads, device="cuda")
        fx.idx_attend_local(q, codes, scales, n_vis, n, 0.02, out, ws, lse=lse, window=window, group=group, pages=pages,
                            page_size=page, seq=s)
        got.append((out, lse))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert torch.isfinite(got[0][1]).all()


def make_plan(pl, g, nseq, group, heads=16, steps=40):
    core = pl.CoreAttention(nseq, 300, nseq * group, heads=heads, k=8, page_size=16)
    layer = pl.LayerAttention(core, window=20, group=group, eps=1e-6,
                              signs=(torch.randint(0, 2, (128,), device="cuda", generator=g) * 2 - 1).to(torch.int8))
    for b in range(nseq):
        core.reserve(b, steps)
        x = torch.randn(steps, 512, device="cuda", generator=g).bfloat16()
        at, seq = torch.arange(steps, device="cuda"), torch.full((steps,), b, dtype=torch.int32, device="cuda")
        layer.write(seq, at, main=x)
        last = slice(steps - layer.ring, steps)
        layer.write(seq[last], at[last], local=x[last])
    return layer


def a_step(layer, g, order, steps=40):
    """q, pos, seq, n_vis, idx and n_local of a step whose runs are of sequences `order`"""
    core, group = layer.core, layer.group
    seq = torch.tensor(order, dtype=torch.int32, device="cuda").repeat_interleave(group)
    pos = (steps - group + torch.arange(group, device="cuda")).repeat(len(order))
    n_vis = (pos + 1).int()
    idx = (torch.rand(core.nq, 8, device="cuda", generator=g) * n_vis[:, None]).int()
    return torch.randn(core.q.shape, device="cuda", generator=g).bfloat16(), pos, seq, n_vis, idx, n_vis.clone()


@pytest.mark.parametrize("group", [1, 3])
def test_on_another_stream(pl, group):
    """the current stream is busy: what the step reads may not come from there"""
    g = torch.Generator(device="cuda").manual_seed(group)
    layer = make_plan(pl, g, 4, group)
    side, big = torch.cuda.Stream(), torch.randn(4096, 4096, device="cuda", generator=g)
    for order in ([2, 0, 3, 1], [1, 3, 0, 2], [0, 0, 1, 1]):
        given = a_step(layer, g, order)
        want = [t.clone() for t in layer.run(*given)]
        layer.out.fill_(7), layer.lse.fill_(7)
        torch.cuda.synchronize()
        for _ in range(8):
            big @ big
        out, lse = layer.run(*given, stream=side)
        with torch.cuda.stream(side):
            got = out.clone(), lse.clone()
        side.synchronize()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("group", [1, 3])
def test_recorded_steps(fx, pl, group):
    """replays read the sequences as they are then, whatever was allocated and freed in between"""
    g = torch.Generator(device="cuda").manual_seed(10 + group)
    layer = make_plan(pl, g, 4, group)
    given = a_step(layer, g, [2, 0, 3, 1])
    with fx.record() as calls:
        layer.run(*given)
    replay = fx.Recorded(calls)
    for order in ([2, 0, 3, 1], [1, 3, 0, 2], [3, 3, 2, 0]):
        for to, x in zip(given, a_step(layer, g, order)):
            to.copy_(x)
        junk = [torch.full((n,), 1, dtype=torch.int32, device="cuda") for n in (1, 4, 12, 64, 100) for _ in range(20)]
        del junk
        replay()
        got = layer.out.clone(), layer.lse.clone()
        layer.out.fill_(7), layer.lse.fill_(7)
        out, lse = layer.run(*given)
        torch.cuda.synchronize()
        assert torch.equal(got[0], out) and torch.equal(got[1], lse)


@pytest.mark.parametrize("format, dim, width, groups", [("main", 512, 256, 32), ("local", 512, 512, 16), ("key", 128, 64, 4)])
@pytest.mark.parametrize("tokens", [1, 9, 700])
def test_kept_rows(fx, format, dim, width, groups, tokens):
    """the tokens that are kept are stored as without the others, and no other row is written"""
    g = torch.Generator(device="cuda").manual_seed(tokens)
    x = torch.randn(tokens, dim, device="cuda", generator=g)
    at = torch.randperm(tokens + 5, device="cuda", generator=g)[:tokens]
    keep = torch.randint(-(1 << 40), 1 << 40, (tokens,), device="cuda", generator=g)
    keep[0] = 0
    if tokens > 1:
        keep[-1] = -1
        at[-1] = at[0]  # an idle slot at a real token's entry
    signs = (torch.randint(0, 2, (128,), device="cuda", generator=g) * 2 - 1).to(torch.int8)
    some = (keep >= 0).nonzero().flatten()
    caches = []
    for rows, places, k in ((x, at, keep), (x[some], at[some], None), (x[some], at[some], at[some])):
        codes = torch.full((tokens + 5, width), 0xA5, dtype=torch.uint8, device="cuda")
        scales = torch.full((tokens + 5, groups), 0xA5, dtype=torch.uint8, device="cuda")
        fx.idx_write_rows(format, rows, codes, scales, places, tokens + 5, eps=1e-6, signs=signs, keep=k)
        caches.append((codes, scales))
    for codes, scales in caches[1:]:
        assert torch.equal(codes, caches[0][0]) and torch.equal(scales, caches[0][1])
    assert (caches[0][0] != 0xA5).any(1).sum() == len(some)


def test_idle_slots_with_positions(pl):
    """a compressed cache: entries and positions differ, and a padded batch's idle slots name positions that live rows of
    their sequence's ring have"""
    g = torch.Generator(device="cuda").manual_seed(0)
    layer = make_plan(pl, g, 3, 2)
    core = layer.core
    before = [t.clone() for t in (core.codes, core.scales, layer.codes, layer.scales, layer.k_codes, layer.k_scales)]
    seq = torch.tensor([0, 0, 1, 2, 2], dtype=torch.int32, device="cuda")
    at = torch.tensor([10, -1, -1, 11, -5], device="cuda")
    pos = torch.tensor([40, 39, 25, 41, 41], device="cuda")
    x, k = torch.randn(5, 512, device="cuda", generator=g), torch.randn(5, 128, device="cuda", generator=g)
    layer.write(seq, at, main=x, local=x, key=k, pos=pos)
    now = (core.codes, core.scales, layer.codes, layer.scales, layer.k_codes, layer.k_scales)
    local = [0 * layer.ring + 40 % layer.ring, 2 * layer.ring + 41 % layer.ring]
    main = [int(core.pages[b, e // 16]) * 16 + e % 16 for b, e in ((0, 10), (2, 11))]
    key = [0 * core.n + 10, 2 * core.n + 11]
    for i, rows in enumerate((main, main, local, local, key, key)):
        changed = (now[i] != before[i]).any(1).nonzero().flatten().tolist()
        assert set(changed) <= set(rows), i  # (a scale may come out as it was)
        if i % 2 == 0:
            assert changed == sorted(rows)
    live = [0, 3]  # and they hold what a call without the idle slots stores
    for t in now:
        t.zero_()
    layer.write(seq, at, main=x, local=x, key=k, pos=pos)
    padded = [t.clone() for t in now]
    for t in now:
        t.zero_()
    layer.write(seq[live], at[live], main=x[live], local=x[live], key=k[live], pos=pos[live])
    for a, b in zip(now, padded):
        assert torch.equal(a, b)


def test_fewer_queries_than_the_plan_has(pl):
    """single queries of different sequences in a plan for draft positions: as in a plan for single queries"""
    g = torch.Generator(device="cuda").manual_seed(5)
    big, one = make_plan(pl, g, 2, 3), make_plan(pl, g, 6, 1)
    # the same rows of two sequences in both
    for layer in (big, one):
        g.manual_seed(6)
        for b in range(2):
            x = torch.randn(40, 512, device="cuda", generator=g).bfloat16()
            at, seq = torch.arange(40, device="cuda"), torch.full((40,), b, dtype=torch.int32, device="cuda")
            layer.write(seq, at, main=x)
            layer.write(seq[-layer.ring:], at[-layer.ring:], local=x[-layer.ring:])
    seq = torch.tensor([0, 1, 1, 1, 0, 1], dtype=torch.int32, device="cuda")
    pos = torch.full((6,), 39, device="cuda")
    n_vis = (pos + 1).int()
    idx = (torch.rand(6, 8, device="cuda", generator=g) * 40).int()
    q = torch.randn(big.core.q.shape, device="cuda", generator=g).bfloat16()
    got = big.run(q, pos, seq, n_vis, idx, n_vis, group=1)
    want = one.run(q, pos, seq, n_vis, idx, n_vis)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.isfinite(got[1]).all()


def test_a_padded_run(pl):
    """a sequence with fewer queries than the step: the padding gives nothing, and what it holds has no effect"""
    g = torch.Generator(device="cuda").manual_seed(7)
    layer = make_plan(pl, g, 3, 3)
    q, pos, seq, n_vis, idx, n_local = a_step(layer, g, [2, 0, 1])
    idle = [4, 5, 8]
    n_vis[idle] = 0
    n_local[idle] = 0
    rest = [t for t in range(9) if t not in idle]
    outs = []
    for _ in range(2):
        out, lse = layer.run(q, pos, seq, n_vis, idx, n_local)
        assert (out[idle] == 0).all() and torch.isneginf(lse[idle]).all()
        outs.append((out[rest].clone(), lse[rest].clone()))
        q[idle], pos[idle], idx[idle] = torch.nan, 7, 3
        seq[idle] = -1
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert torch.isfinite(outs[0][1]).all()
