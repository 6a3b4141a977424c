"""What LayerAttention gives to the library's calls, and its refusals (no GPU: the calls are looked at, not made)."""
import pytest
import torch

from test_abi import call, fx  # noqa: F401
from test_operator_args import refuse
from test_rows_args import L, LOCAL


@pytest.fixture
def calls(monkeypatch):
    """(pipeline, a list that the calls' names and arguments are put into)"""
    from top_fp4_lightning_amd import pipeline

    made = []
    for name in ("idx_rope", "idx_attend", "idx_attend_local", "idx_write_rows"):
        monkeypatch.setattr(pipeline, name, lambda *a, _name=name, **k: made.append((_name, a, k)))
    return pipeline, made


def plan(pl, nseq, group, **kw):
    core = pl.CoreAttention(nseq, 40, nseq * group, heads=2, k=4, page_size=16, device="cpu")
    return pl.LayerAttention(core, window=8, group=group, **kw)


def step(layer, seq):
    nq = layer.core.nq
    ints = torch.zeros(nq, dtype=torch.int32)
    return layer.core.q.clone(), torch.zeros(nq, dtype=torch.int64), seq, ints, torch.zeros(nq, 4, dtype=torch.int32), ints + 1


def storage(t):
    return t.untyped_storage().data_ptr()


@pytest.mark.parametrize("group", [1, 3])
def test_a_step_makes_no_tensors(calls, group):
    """a recorded step keeps addresses, and one on another stream may not read what the current stream is writing: every
    tensor of its calls is the caller's or the plan's"""
    pl, made = calls
    layer = plan(pl, 4, group)
    given = step(layer, torch.tensor([2, 0, 3, 1], dtype=torch.int32).repeat_interleave(group))
    layer.run(*given)
    kept = {storage(t) for t in [*given, *vars(layer).values(), *vars(layer.core).values()] if isinstance(t, torch.Tensor)}
    for name, args, kw in made:
        for t in [*args, *kw.values()]:
            assert not isinstance(t, torch.Tensor) or storage(t) in kept, name
    local = [kw for name, _, kw in made if name == "idx_attend_local"]
    assert [kw["seq"].tolist() for kw in local] == [[2, 0, 3, 1]] and local[0]["group"] == group


def test_strided_refusals(fx):
    good = [*LOCAL[:13], 3, *LOCAL[13:]]
    name = "idx_attend_local_strided"
    refuse(fx, name, good, [(13, -1, fx.IDX_EINVAL)])
    refuse(fx, name, good, [(i + (i > 12), None, fx.IDX_EINVAL) for i in (L["q"], L["n_vis"], L["out"], L["base"])])
    none = list(good)
    none[L["nq"]] = 0
    assert call(fx, name, *none)[0] == fx.IDX_OK


def test_binding_refuses_other_views(fx):
    q, codes = torch.zeros(6, 2, 512, dtype=torch.bfloat16), torch.zeros(10, 512, dtype=torch.uint8)
    pages = torch.zeros(3, 1, dtype=torch.int32)
    seq = torch.zeros(6, dtype=torch.int32)
    for bad, error in ((seq, ValueError), (seq[:4:2], ValueError), (seq.long()[::2], TypeError), (seq[::2].view(3, 1), ValueError),
                       (seq[::2], ValueError)):  # the last: not on a GPU
        with pytest.raises(error):
            fx.idx_attend_local(q, codes, torch.zeros(10, 16, dtype=torch.uint8), torch.zeros(6, dtype=torch.int32), 10, 1.0,
                                q.clone(), torch.zeros(16, dtype=torch.uint8), group=2, pages=pages, page_size=10, seq=bad)
