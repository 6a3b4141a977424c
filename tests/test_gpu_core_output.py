"""The core attention's output as a layer gives it on: a cache row is key and value at once, so the values that carry
the rotary position have to be turned back, and the factor that goes with stretched frequencies taken out."""
import numpy as np
import pytest
import torch

import attn_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pl():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from top_fp4_lightning_amd import pipeline

    return pipeline


def turned_back(o, pos, freq, mscale, layout):
    """o [heads, 512] in 64 bits, its last 2 len(freq) values turned by -pos * freq and divided by mscale"""
    rot = 2 * len(freq)
    z = np.exp(-1j * float(pos) * freq) / mscale
    y, part = o.copy(), o[:, 512 - rot:]
    x = part[:, :rot // 2] + 1j * part[:, rot // 2:] if layout == "half" else part[:, 0::2] + 1j * part[:, 1::2]
    x = x * z
    if layout == "half":
        y[:, 512 - rot:] = np.concatenate([x.real, x.imag], 1)
    else:
        y[:, 512 - rot::2], y[:, 513 - rot::2] = x.real, x.imag
    return y


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("stretch", [{}, dict(scaling="yarn", factor=4.0, original=1024.0)])
def test_output_against_the_definition(pl, layout, stretch):
    """the rows that the cache holds, averaged and turned back in 64 bits. Tolerance: the attention's own (its result
    is rounded to bf16) of both values of a pair, and the second rounding, half a step; the turn's fp32 2^-20."""
    n, heads, k = 900, 20, 200
    core = pl.CoreAttention(2, n, 3, heads=heads, k=k, page_size=48, layout=layout, **stretch)
    g = torch.Generator(device="cuda").manual_seed(3)
    for b in range(2):
        core.write(b, 0, torch.randn(n, 512, device="cuda", generator=g).bfloat16())
    q = (2.0 * torch.randn(3, heads, 512, device="cuda", generator=g)).bfloat16()
    pos = torch.tensor([899, 500, 77], device="cuda")
    seq = torch.tensor([0, 1, 1], dtype=torch.int32, device="cuda")
    nv = (pos + 1).int()
    idx = torch.stack([torch.randperm(900, device="cuda", generator=g)[:k] for _ in range(3)]).int()
    out, lse = core.layer(q, pos, seq, nv, idx)
    torch.cuda.synchronize()
    freq = core.freq.cpu().numpy()
    codes, scales, pages = core.codes.cpu().numpy(), core.scales.cpu().numpy(), core.pages.cpu().numpy()
    for t in range(3):
        _, rows = ref.entries(t, nv.tolist(), n, len(codes), pages=pages, page_size=48, seq=seq.tolist(),
                              idx=idx.cpu().numpy())
        r = ref.attention(core.q[t].double().cpu().numpy(), codes, scales, core.scale, rows)
        want = turned_back(r["out"], pos[t], freq, core.mscale, layout)
        tol = ref.out_tolerance(r, len(rows))
        pair = np.abs(turned_back(tol, 0, freq, core.mscale, layout))  # (the place's own over mscale)
        other = pair.copy()
        if layout == "half":
            other[:, 448:] = np.roll(pair[:, 448:], 32, axis=1)
        else:
            other[:, 448:] = pair[:, 448:].reshape(heads, 32, 2)[:, :, ::-1].reshape(heads, 64)
        size = np.abs(want) + 2.0 ** -20 * np.abs(r["out"]).max()
        tol = np.where(np.arange(512) < 448, tol, pair + other + 2.0 ** -8 * (size + pair + other))
        err = np.abs(out[t].double().cpu().numpy() - want)
        assert (err <= tol).all(), (t, err.max())
        assert (np.abs(lse[t].double().cpu().numpy() - r["lse"]) <= ref.lse_tolerance(r, len(rows))).all()


def test_output_is_in_the_rows_units(pl):
    """A query of zeros at the position of its only entry: the output is that row, wherever it stands, with every
    scaling. Bound: the stored value of a group of 16 is off by half of the widest step (4 .. 6: 1) times the scale,
    which is at most 2^-3 above a sixth of the largest (E4M3's step), so 0.1875 of the largest; rotated values are at
    most sqrt 2 of the group's largest x, both of a pair are off, so 0.1875 * 2 of it. Roundings to bf16, 2^-8 of a
    value: of the turned row (2 * 2^-8 of the largest after the way back), of the average, whose values are up to
    0.1875 larger (2 * 1.1875 * 2^-8), of the result (1.375 * 2^-8 * sqrt 2): below 0.03 together."""
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(700, 512, device="cuda", generator=g).bfloat16()
    bound = x[:, 448:].float().abs().view(-1, 4, 16).amax(-1).repeat_interleave(16, 1) * (0.375 + 0.03)
    for stretch in ({}, dict(scaling="yarn", factor=4.0, original=64.0), dict(scaling="linear", factor=8.0)):
        core = pl.CoreAttention(1, 700, 700, heads=2, k=1, page_size=64, **stretch)
        core.write(0, 0, x)
        q = torch.zeros(700, 2, 512, dtype=torch.bfloat16, device="cuda")
        pos = torch.arange(700, device="cuda")
        seq = torch.zeros(700, dtype=torch.int32, device="cuda")
        out, _ = core.layer(q, pos, seq, (pos + 1).int(), pos.int()[:, None])
        assert ((out[:, :, 448:].float() - x[:, None, 448:].float()).abs() <= bound[:, None]).all(), stretch
        raw, _ = core.run(q, pos, seq, (pos + 1).int(), pos.int()[:, None])
        assert ((raw[:, :, 448:].float() - x[:, None, 448:].float()).abs() > bound[:, None]).any()  # in the cache's frame


def test_a_captured_layer_replays(pl):
    g = torch.Generator(device="cuda").manual_seed(5)
    core = pl.CoreAttention(1, 3000, 2, heads=64, k=512, page_size=64, scaling="yarn", factor=4.0, original=1024.0)
    core.write(0, 0, torch.randn(3000, 512, device="cuda", generator=g).bfloat16())
    q = torch.randn(2, 64, 512, device="cuda", generator=g).bfloat16()
    pos = torch.tensor([2998, 2999], device="cuda")
    seq = torch.zeros(2, dtype=torch.int32, device="cuda")
    nv = (pos + 1).int()
    idx = torch.stack([torch.randperm(2999, device="cuda", generator=g)[:512] for _ in range(2)]).int()
    want = [v.clone() for v in core.layer(q, pos, seq, nv, idx)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        core.layer(q, pos, seq, nv, idx)
    for rep in range(3):
        core.out.zero_()
        core.lse.zero_()
        (torch.randn(64, 64, device="cuda") @ torch.randn(64, 64, device="cuda")).sum()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(core.out, want[0]) and torch.equal(core.lse, want[1]), rep


def test_parts_of_a_selection_join_by_their_lse(pl):
    """attention over two halves of a selection, joined in the cache's frame and turned back, is attention over it all:
    three roundings to bf16 of averages whose sizes add up to at most sum p |kv|, with the logits' own error"""
    g = torch.Generator(device="cuda").manual_seed(6)
    core = pl.CoreAttention(1, 2000, 5, heads=20, k=300, page_size=64, scaling="yarn", factor=4.0, original=256.0)
    core.write(0, 0, torch.randn(2000, 512, device="cuda", generator=g).bfloat16())
    q = (2.0 * torch.randn(5, 20, 512, device="cuda", generator=g)).bfloat16()
    pos = torch.arange(1995, 2000, device="cuda")
    seq = torch.zeros(5, dtype=torch.int32, device="cuda")
    nv = (pos + 1).int()
    idx = torch.stack([torch.randperm(1990, device="cuda", generator=g)[:300] for _ in range(5)]).int()
    parts = []
    for lst in (idx[:, :100], idx[:, 100:]):
        out, lse = core.run(q, pos, seq, nv, lst)
        parts.append((out.double(), lse.double().clone()))
    lse = torch.logaddexp(parts[0][1], parts[1][1])
    joined = sum(o * (l - lse).exp()[:, :, None] for o, l in parts)
    whole, whole_lse = core.run(q, pos, seq, nv, idx)
    codes, scales, pages = core.codes.cpu().numpy(), core.scales.cpu().numpy(), core.pages.cpu().numpy()
    for t in range(5):
        _, rows = ref.entries(t, nv.tolist(), 2000, len(codes), pages=pages, page_size=64, seq=[0] * 5, idx=idx.cpu().numpy())
        r = ref.attention(core.q[t].double().cpu().numpy(), codes, scales, core.scale, rows)
        tol = 3 * ref.out_tolerance(r, 300) + 2 * 2.0 ** -8 * r["A"]
        assert (np.abs((joined[t] - whole[t].double()).cpu().numpy()) <= tol).all(), t
        assert (np.abs((lse[t] - whole_lse[t].double()).cpu().numpy()) <= 3 * ref.lse_tolerance(r, 300)).all(), t
