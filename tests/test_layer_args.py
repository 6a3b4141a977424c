"""What LayerAttention gives to the library's calls, and its refusals (no GPU: the calls are looked at, not made)."""
import pytest
import torch

import rows_ref
from test_abi import FAKE, call, fx  # noqa: F401
from test_operator_args import refuse
from test_rows_args import L, LOCAL, W, WRITE


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


def written(args, kw, max_n, rows):
    """{token: cache row} of a call, by the definition"""
    at, keep = kw["at"], kw.get("keep")
    where = dict(pages=kw["pages"].numpy(), page_size=kw["page_size"], seq=kw["seq"].numpy(), ring=kw.get("ring", 0))
    found = {t: rows_ref.row_of(t, at, max_n, rows, **where) for t in range(len(at)) if keep is None or keep[t] >= 0}
    return {t: r for t, r in found.items() if r >= 0}


@pytest.mark.parametrize("compressed", [False, True])
def test_tokens_that_are_left_out(calls, compressed):
    """a token at an entry below 0 is written to none of the caches, with or without positions of its own"""
    pl, made = calls
    layer = plan(pl, 3, 1, signs=torch.ones(128, dtype=torch.int8))
    for b in range(3):
        layer.core.reserve(b, 20)
    at = torch.tensor([5, -1, 7, -1, 0])
    pos = torch.tensor([20, 20, 29, 0, 3]) if compressed else None  # (an idle slot may name a real token's position)
    seq = torch.tensor([0, 0, 1, 2, 2], dtype=torch.int32)
    x = torch.zeros(5, 512)
    layer.write(seq, at, main=x, local=x, key=x[:, :128], pos=pos)
    rows = dict(main=len(layer.core.codes), local=len(layer.codes), key=len(layer.k_codes))
    assert [args[0] for _, args, _ in made] == ["main", "local", "key"]
    for _, args, kw in made:
        kw["at"], max_n = args[4], args[5]
        assert sorted(written(args, kw, max_n, rows[args[0]])) == [0, 2, 4], args[0]
        assert args[0] != "local" or torch.equal(kw["at"], at if pos is None else pos)


def test_kept_refusals(fx):
    good = [*WRITE[:-1], FAKE, None]
    refuse(fx, "idx_write_rows_kept", good, [(27, FAKE + 4, fx.IDX_EALIGN), (W["x"], None, fx.IDX_EINVAL),
                                             (W["eps"], 0.0, fx.IDX_EINVAL), (W["format"], 3, fx.IDX_EUNSUPPORTED)])
    codes, at = torch.zeros(10, 512, dtype=torch.uint8), torch.zeros(3, dtype=torch.int64)
    for keep, error in ((at[:2], ValueError), (at.int(), TypeError), (at.repeat(2)[::2], ValueError), (at, ValueError)):
        with pytest.raises(error):  # (the last: not on a GPU)
            fx.idx_write_rows("local", torch.zeros(3, 512), codes, codes[:, :16].contiguous(), at, 10, keep=keep)


def test_queries_of_a_step(calls):
    """a plan for three draft positions takes steps of fewer: every query goes to its own sequence's ring"""
    pl, made = calls
    layer = plan(pl, 2, 3)
    seq = torch.tensor([1, 0, 1, 1, 0, 0], dtype=torch.int32)
    for group in (1, 2, 3, None):
        layer.run(*step(layer, seq), group=group)
        kw = made[-1][2]
        assert kw["group"] == (group or 3) and kw["seq"].tolist() == seq[::kw["group"]].tolist()
    made.clear()
    for group in (0, 4, -1):
        with pytest.raises(ValueError):
            layer.run(*step(layer, seq), group=group)
    assert not made


def test_keys_of_a_plan_without_signs(calls):
    pl, made = calls
    layer = plan(pl, 2, 1)
    at, x = torch.zeros(2, dtype=torch.int64), torch.zeros(2, 512)
    with pytest.raises(ValueError, match="signs"):
        layer.write(at.int(), at, main=x, local=x, key=x[:, :128])
    assert not made  # before anything is written
