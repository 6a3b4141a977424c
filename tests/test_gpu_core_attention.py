"""The operators together, as a model uses them: rows rotated and quantised into pages, a layer's selection, core
attention over it, and the training signal for the layer's scores."""
import numpy as np
import pytest
import torch

import attn_ref as ref
import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pl():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from top_fp4_lightning_amd import pipeline

    return pipeline


def rotated(x, pos, freq, mscale):
    """the last 2 len(freq) values of rows x [m, heads, 512] rotated by interleaved pairs, in 64 bits"""
    a = np.asarray(pos, np.float64)[:, None] * freq
    z = x[..., 512 - 2 * len(freq):].reshape(*x.shape[:-1], -1, 2)
    z = (z[..., 0] + 1j * z[..., 1]) * (mscale * np.exp(1j * a))[:, None]
    y = x.copy()
    y[..., 512 - 2 * len(freq):] = np.stack([z.real, z.imag], -1).reshape(*x.shape[:-1], -1)
    return y


def setup(pl, lens, heads=64, layers=1, write_mask=True):
    wl = synth.decode_workload("core", 55, lens, layers=layers)
    dev = pl.DeviceWorkload.from_workload(wl)
    plan = pl.MaskFormPlan(dev, k=512, write_mask=write_mask).run()
    nq, n = dev.nq, max(lens)
    core = pl.CoreAttention(nq, n, nq, heads=heads, page_size=48, scaling="yarn", factor=4.0, original=1024.0)
    g = torch.Generator(device="cuda").manual_seed(56)
    rows = []
    order = [(b, f) for b in range(nq) for f in range(0, lens[b], 1500)]
    for b, f in sorted(order, key=lambda x: x[1]):  # the sequences grow in turn: their pages are mixed
        m = min(1500, lens[b] - f)
        x = torch.randn(m, 512, device="cuda", generator=g).bfloat16()
        core.write(b, f, x)
        rows.append((b, f, x))
    q = (2.0 * torch.randn(nq, heads, 512, device="cuda", generator=g)).bfloat16()
    pos = torch.tensor([x - 1 for x in lens], device="cuda")
    seq = torch.arange(nq, dtype=torch.int32, device="cuda")
    return plan, core, q, pos, seq, rows


def test_attention_over_the_selection_of_a_layer(pl):
    from top_fp4_lightning_amd import idx_gather_kv

    lens = [5000, 700, 3210]
    plan, core, q, pos, seq, _ = setup(pl, lens)
    dv = plan.dev
    for layer in range(plan.L):
        idx = plan.layer_topk(layer)[0]  # rows at a stride
        out, lse = core.run(q, pos, seq, dv.n_vis, idx)
        w = core.selection_weights(seq, dv.n_vis, idx)
        torch.cuda.synchronize()
        # the query that was rotated is within a bf16 rounding of the rotation
        want_q = rotated(q.double().cpu().numpy(), pos.cpu().numpy(), core.freq.cpu().numpy(), core.mscale)
        got_q = core.q.double().cpu().numpy()
        assert (np.abs(got_q - want_q) <= 2.0 ** -8 * np.abs(want_q) + 2.0 ** -18).all()
        pages, sel = core.pages.cpu().numpy(), idx.cpu().numpy()
        codes, scales = core.codes.cpu().numpy(), core.scales.cpu().numpy()
        for t, n in enumerate(lens):
            assert sorted(sel[t][sel[t] >= 0]) == list(sel[t][sel[t] >= 0]) and (sel[t] >= 0).sum() == min(n, 512)
            slots, rows = ref.entries(t, lens, max(lens), len(codes), pages=pages, page_size=48, seq=seq.cpu().numpy(), idx=sel)
            r = ref.attention(got_q[t], codes, scales, core.scale, rows)
            assert (np.abs(out[t].double().cpu().numpy() - r["out"]) <= ref.out_tolerance(r, len(rows))).all(), (layer, t)
            assert (np.abs(lse[t].double().cpu().numpy() - r["lse"]) <= ref.lse_tolerance(r, len(rows))).all()
            x = r["p"].mean(0)
            got_w = w[t].double().cpu().numpy()
            # from a lse good to its tolerance
            tol = ref.weight_tolerance(r, x) + x * 1.05 * ref.lse_tolerance(r, len(rows)).max()
            assert (np.abs(got_w[slots] - x) <= tol).all()
            # the rows that idx_gather_kv copies out are those that were attended to
            base = torch.zeros(1, dtype=torch.int64, device="cuda")
            flat = torch.full((1, 512), -1, dtype=torch.int32, device="cuda")
            flat[0, :len(rows)] = torch.tensor(rows, dtype=torch.int32, device="cuda")
            kv = idx_gather_kv(core.codes, core.scales, base, torch.full((1,), len(codes), dtype=torch.int32, device="cuda"), flat)
            assert np.array_equal(kv[0, :len(rows)].double().cpu().numpy(), ref.kv_rows(codes[rows], scales[rows]))


def test_training_signal_of_the_indexer(pl):
    lens = [4000, 600, 2500]
    plan, core, q, pos, seq, _ = setup(pl, lens)
    dis = pl.IndexerDistill(plan, core)
    n_vis = plan.dev.n_vis.cpu().numpy()
    for layer in range(plan.L):
        loss, grad = dis.run(layer, q, pos, seq)
        torch.cuda.synchronize()
        s = plan.scores.view(3, plan.L, -1)[:, layer].double().cpu().numpy()
        w = core.weights.double().cpu().numpy()
        idx = dis.idx.cpu().numpy()
        for t, n in enumerate(n_vis):
            p = np.zeros(n)
            live = idx[t] >= 0
            p[idx[t][live]] = w[t][live] / w[t][live].sum()
            x = s[t, :n]
            lq = x - (x.max() + np.log(np.exp(x - x.max()).sum()))
            # log w is good to 2^-22 of itself (below 64) and the rest to fp32's exponentials: see test_gpu_distill.py
            big = np.abs(x[np.isfinite(x)]).max() + 64
            hit = p > 0
            want = (p[hit] * (np.log(p[hit]) - lq[hit])).sum()
            assert abs(float(loss[t]) - want) <= 2.0 ** -20 * (2 + big), (layer, t)
            g = (np.exp(lq) - p) / 3
            tol = (np.exp(lq) + p) / 3 * 2.0 ** -19 * (2 + big) + 2.0 ** -125
            assert (np.abs(grad[t, :n].double().cpu().numpy() - g) <= tol).all(), (layer, t)
            assert (grad[t, :n][torch.isneginf(plan.scores.view(3, plan.L, -1)[t, layer, :n])] == 0).all()


def test_a_captured_step_replays(pl):
    lens = [3000, 900]
    plan, core, q, pos, seq, _ = setup(pl, lens)
    dis = pl.IndexerDistill(plan, core)
    eager = [x.clone() for x in dis.run(1, q, pos, seq)] + [core.out.clone(), core.weights.clone()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dis.run(1, q, pos, seq)
    for rep in range(3):
        for x in (dis.loss, dis.dscores, core.out, core.weights):
            x.zero_()
        (torch.randn(64, 64, device="cuda") @ torch.randn(64, 64, device="cuda")).sum()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, (dis.loss, dis.dscores, core.out, core.weights)):
            assert torch.equal(a, b), rep
    # other queries in the captured buffer: the replay follows them
    q.copy_(q.flip(1))
    graph.replay()
    torch.cuda.synchronize()
    got = [x.clone() for x in (dis.loss, dis.dscores, core.out, core.weights)]
    dis.run(1, q, pos, seq)
    torch.cuda.synchronize()
    for a, b in zip(got, (dis.loss, dis.dscores, core.out, core.weights)):
        assert torch.equal(a, b)


def test_rows_outside_the_sequence_are_refused(pl):
    core = pl.CoreAttention(1, 100, 1, page_size=16)
    x = torch.zeros(10, 512, dtype=torch.bfloat16, device="cuda")
    for first in (-1, 91):
        with pytest.raises(ValueError):
            core.write(0, first, x)
    core.write(0, 90, x)
    assert core.given == [7] and (core.pages >= 0).sum() == 7
