"""Rows written into CoreAttention's pages: the positions that turn them, and refusals that leave the cache as it was."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pl():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from top_fp4_lightning_amd import pipeline

    return pipeline


def stored(core, b, first, m):
    at = torch.arange(first, first + m, device="cuda")
    rows = core.pages[b].long()[at // core.page_size] * core.page_size + at % core.page_size
    return core.codes[rows], core.scales[rows]


def test_entries_at_positions_of_their_own(pl):
    """entries that stand for two tokens each, turned by the second's position; by default entry i stands at i"""
    from top_fp4_lightning_amd import idx_quantize_kv, idx_rope

    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(300, 512, device="cuda", generator=g).bfloat16()
    core = pl.CoreAttention(2, 400, 1, heads=4, k=8, page_size=24)
    for first, part in ((0, slice(0, 100)), (100, slice(100, 101)), (101, slice(101, 300))):
        core.write(0, first, x[part], pos=2 * torch.arange(300, device="cuda")[part] + 1)
        core.write(1, first, x[part])
    for b, pos in ((0, 2 * torch.arange(300, device="cuda") + 1), (1, torch.arange(300, device="cuda"))):
        y = idx_rope(x.view(300, 1, 512), pos, core.freq, layout=core.layout, mscale=core.mscale)
        for got, want in zip(stored(core, b, 0, 300), idx_quantize_kv(y.view(300, 512))):
            assert torch.equal(got, want), b


def test_refused_rows_leave_the_cache(pl):
    core = pl.CoreAttention(1, 100, 1, heads=4, k=8, page_size=16)
    x = torch.randn(10, 512, device="cuda").bfloat16()
    core.write(0, 0, x)
    before = [t.clone() for t in (core.codes, core.scales, core.pages)] + [list(core.given), core.used]
    pos = torch.arange(10, device="cuda")
    for bad, err in ((dict(x=x.float()), TypeError), (dict(x=x.cpu()), ValueError), (dict(pos=pos[:9]), ValueError),
                     (dict(pos=pos.int()), TypeError), (dict(first=91), ValueError)):
        with pytest.raises(err):
            core.write(**{**dict(b=0, first=60, x=x, pos=pos), **bad})
    core.write(0, 40, x[:0])  # no rows
    after = [core.codes, core.scales, core.pages, core.given, core.used]
    assert all(torch.equal(a, b) for a, b in zip(before[:3], after[:3])) and before[3:] == after[3:]
