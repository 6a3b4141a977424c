"""A layer's attention as a decode step runs it: rows of all three caches written, the queries turned, the selection and
the local positions attended to and joined. Captured once and replayed, against 64-bit definitions from the rows given."""
import numpy as np
import pytest
import torch

import local_ref
import rows_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pl():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from top_fp4_lightning_amd import pipeline

    return pipeline


def f64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("group, layout, freqs", [(1, "interleaved", dict(scaling="yarn", factor=8.0)), (1, "half", {}),
                                                  (3, "interleaved", dict(scaling="yarn", factor=4.0))])
def test_decode_steps(pl, group, layout, freqs):
    nseq, n, heads, k, window, steps = 3, 300, 24, 40, 20, 34
    nq = nseq * group
    g = torch.Generator(device="cuda").manual_seed(group)
    gamma = torch.rand(512, device="cuda", generator=g) + 0.5
    signs = (torch.randint(0, 2, (128,), device="cuda", generator=g) * 2 - 1).to(torch.int8)
    core = pl.CoreAttention(nseq, n, nq, heads=heads, k=k, page_size=16, layout=layout, **freqs)
    layer = pl.LayerAttention(core, window=window, group=group, signs=signs, gamma=gamma, eps=1e-5)
    for b in range(nseq):
        core.reserve(b, 100 + steps * group + 5 * b)
    first = torch.tensor([0, 57, 3], device="cuda")  # positions that the sequences start at
    pos = torch.empty(nq, dtype=torch.int64, device="cuda")
    seq = torch.arange(nseq, device="cuda").repeat_interleave(group).int()
    main, local = (torch.empty(nq, 512, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    key = torch.empty(nq, 128, dtype=torch.bfloat16, device="cuda")
    q = torch.empty(nq, heads, 512, dtype=torch.bfloat16, device="cuda")
    n_vis = torch.empty(nq, dtype=torch.int32, device="cuda")
    idx = torch.empty(nq, k, dtype=torch.int32, device="cuda")

    def step():
        layer.write(seq, pos, main=main, local=local, key=key)
        layer.run(q, pos, seq, n_vis, idx, n_vis)

    def fill(i):
        pos.copy_((first[:, None] + i * group + torch.arange(group, device="cuda")).reshape(-1))
        n_vis.copy_(pos + 1)
        for x in (main, local, key, q):
            x.copy_(torch.randn(x.shape, device="cuda", generator=g))
        idx.copy_((torch.rand(nq, k, device="cuda", generator=g) * n_vis[:, None]).int())
        idx[:, k // 2:] = torch.where(torch.rand(nq, k - k // 2, device="cuda", generator=g) < 0.3, -1, idx[:, k // 2:])

    fill(0)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        step()
    freq, m = core.freq.cpu().numpy(), core.mscale
    stored = [{} for _ in range(nseq)]  # position -> the main and local rows, as the caches hold them
    for i in range(steps):
        fill(i)
        graph.replay()
        torch.cuda.synchronize()
        p = pos.cpu().numpy()
        turn = (p, freq, 448, layout, m)
        rows = [rows_ref.quantise(f, rows_ref.rotate(rows_ref.normalise(f64(x), f64(gamma), 1e-5), *turn))
                for f, x in (("main", main), ("local", local))]
        keys = rows_ref.quantise("key", rows_ref.transform(rows_ref.rotate(f64(key), p, freq, 64, layout, m), f64(signs)))
        for t in range(nq):
            stored[t // group][int(p[t])] = [rows_ref.values(f, c[t:t + 1], s[t:t + 1])[0]
                                             for f, (c, s) in zip(("main", "local"), rows)]
        at = seq.long().cpu().numpy() * n + p
        assert np.array_equal(layer.k_codes.cpu().numpy()[at], keys[0])
        assert np.array_equal(layer.k_scales.cpu().numpy()[at], keys[1])
        if i not in (0, 1, 9, steps - 1):
            continue
        turned, out, lse = f64(core.q), f64(layer.out), f64(layer.lse)
        for t in range(nq):
            mine = stored[t // group]
            picked = [mine[x][0] for x in idx[t].tolist() if 0 <= x <= p[t] and x in mine]
            # (positions before a sequence's start were never written: zeros)
            picked += [np.zeros(512) for x in idx[t].tolist() if 0 <= x <= p[t] and x not in mine]
            near = [mine[x][1] if x in mine else np.zeros(512) for x in range(max(0, p[t] + 1 - window), p[t] + 1)]
            picked, near = np.array(picked).reshape(-1, 512), np.array(near)
            # the selection's part: its output is rounded to bf16 on the way, half a step
            o1, l1, e1, el1 = local_ref.query(turned[t], picked, core.scale)
            want, l, eo, el = local_ref.query(turned[t], near, core.scale, o1, l1, (p[t], freq, 448, layout, 1 / m))
            share = np.exp(l1 - l)[:, None]
            slack = share * (e1 + el1[:, None] * (np.abs(o1) + np.abs(want).max()))
            pairs = slack.copy()
            h = 32
            i0 = 448 + (np.arange(h) if layout == "half" else 2 * np.arange(h))
            i1 = i0 + (h if layout == "half" else 1)
            pairs[:, i0] = pairs[:, i1] = (slack[:, i0] + slack[:, i1]) / m
            assert (np.abs(out[t] - want) <= eo + pairs).all(), (i, t, (np.abs(out[t] - want) - eo - pairs).max())
            assert (np.abs(lse[t] - l) <= el + el1).all(), (i, t)


def test_the_parts_make_the_whole(pl):
    """the joined result is what one softmax over both parts' entries gives, and each part's weight its share"""
    core = pl.CoreAttention(1, 64, 1, heads=4, k=8, rot=64)
    layer = pl.LayerAttention(core, window=6)
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(30, 512, device="cuda", generator=g).bfloat16()
    core.reserve(0, 30)
    at = torch.arange(30, device="cuda")
    seq = torch.zeros(30, dtype=torch.int32, device="cuda")
    layer.write(seq, at, main=x)
    layer.write(seq[-6:], at[-6:], local=x[-6:])
    q = torch.randn(1, 4, 512, device="cuda", generator=g).bfloat16()
    pos, nv = at[-1:], torch.tensor([30], dtype=torch.int32, device="cuda")
    none = torch.full((1, 8), -1, dtype=torch.int32, device="cuda")
    some = torch.arange(8, dtype=torch.int32, device="cuda").view(1, 8)
    lses = {}
    for name, idx, n_local in (("local", none, nv), ("selected", some, nv * 0), ("both", some, nv), ("none", none, nv * 0)):
        out, lse = layer.run(q, pos, seq[:1], nv, idx, n_local)
        lses[name] = (out.double(), lse.double())
    assert torch.isneginf(lses["none"][1]).all() and (lses["none"][0] == 0).all()
    both = torch.logaddexp(lses["local"][1], lses["selected"][1])
    assert (both - lses["both"][1]).abs().max() < 1e-5
    w = [(lses[k][1] - both).exp()[..., None] for k in ("local", "selected")]
    want = w[0] * lses["local"][0] + w[1] * lses["selected"][0]
    # each part and the whole rounded to bf16: half a step each
    slack = 2.0 ** -8 * (w[0] * lses["local"][0].abs() + 2 * w[1] * lses["selected"][0].abs() + want.abs()) + 2.0 ** -12
    assert ((want - lses["both"][0]).abs() <= slack).all()


def test_reserved_pages(pl):
    core = pl.CoreAttention(2, 100, 1, page_size=16)
    core.reserve(0, 40)
    core.reserve(1, 1)
    core.reserve(0, 41)
    core.reserve(0, 49)
    assert core.pages.tolist() == [[0, 1, 2, 4, -1, -1, -1], [3, -1, -1, -1, -1, -1, -1]]
    with pytest.raises(ValueError):
        core.reserve(0, 101)
    layer = pl.LayerAttention(core, window=8)
    x, at = torch.ones(2, 512, device="cuda"), torch.tensor([48, 64], device="cuda")
    layer.write(torch.zeros(2, dtype=torch.int32, device="cuda"), at, main=x)  # the second has no page: left out
    assert core.codes.any(1).nonzero().flatten().tolist() == [4 * 16]
