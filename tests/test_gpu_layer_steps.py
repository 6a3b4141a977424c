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
