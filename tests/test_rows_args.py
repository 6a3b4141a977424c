"""Argument checks of the calls on rows at places, before any HIP call (no GPU), and the reference of their tests against
plain statements of the formats."""
import math

import numpy as np
import pytest
import torch

import rows_ref as ref
from test_abi import FAKE, call, fx  # noqa: F401
from test_operator_args import refuse

NAN, INF = math.nan, math.inf
# idx_write_rows: format, x, dtype, tokens, x_stride, norm, gamma, eps, pos, freq, rot, offset, layout, mscale, signs, codes,
# scales, rows, kv_base, pages, pages_stride, nseq, page_size, seq, at, max_n, ring, stream
WRITE = [0, FAKE, 0, 4, 512, 1, FAKE, 1e-6, FAKE, FAKE, 64, 448, 1, 1.0, FAKE, FAKE, FAKE, 100, FAKE, None, 0, 0, 0, None,
         FAKE, 100, 0, None]
W = dict(format=0, x=1, dtype=2, tokens=3, stride=4, norm=5, gamma=6, eps=7, pos=8, freq=9, rot=10, offset=11, layout=12,
         mscale=13, signs=14, codes=15, scales=16, rows=17, base=18, pages=19, pstride=20, nseq=21, psize=22, seq=23, at=24,
         max_n=25, ring=26)
# idx_read_rows: format, codes, scales, rows, kv_base, pages, pages_stride, nseq, page_size, seq, at, max_n, ring, tokens,
# pos, freq, rot, offset, layout, mscale, inverse, out, dtype, out_stride, stream
READ = [0, FAKE, FAKE, 100, FAKE, None, 0, 0, 0, None, FAKE, 100, 0, 4, FAKE, FAKE, 64, 448, 1, 1.0, 1, FAKE, 0, 512, None]
R = dict(format=0, codes=1, scales=2, rows=3, base=4, pages=5, pstride=6, nseq=7, psize=8, seq=9, at=10, max_n=11, ring=12,
         tokens=13, pos=14, freq=15, rot=16, offset=17, layout=18, mscale=19, x=21, dtype=22, stride=23)


@pytest.mark.parametrize("name, good, at", [("idx_write_rows", WRITE, W), ("idx_read_rows", READ, R)])
def test_refusals(fx, name, good, at):
    a = at
    none = list(good)
    none[a["tokens"]] = 0
    none[a["x"]] = none[a["at"]] = None
    assert call(fx, name, *none)[0] == fx.IDX_OK
    paged = (a["base"], a["pages"], a["psize"], a["pstride"], a["nseq"])
    refuse(fx, name, good, [
        (a["x"], None, fx.IDX_EINVAL), (a["at"], None, fx.IDX_EINVAL), (a["codes"], None, fx.IDX_EINVAL),
        (a["scales"], None, fx.IDX_EINVAL), (a["pages"], FAKE, fx.IDX_EINVAL),
        (a["format"], 3, fx.IDX_EUNSUPPORTED), (a["format"], -1, fx.IDX_EUNSUPPORTED), (a["dtype"], 2, fx.IDX_EUNSUPPORTED),
        (a["tokens"], -1, fx.IDX_EUNSUPPORTED), (a["tokens"], 1 << 24, fx.IDX_EUNSUPPORTED),
        (a["rows"], -1, fx.IDX_EUNSUPPORTED), (a["max_n"], -1, fx.IDX_EUNSUPPORTED),
        (a["max_n"], (1 << 30) + 1, fx.IDX_EUNSUPPORTED), (a["ring"], -1, fx.IDX_EUNSUPPORTED),
        (a["ring"], (1 << 30) + 1, fx.IDX_EUNSUPPORTED), (a["stride"], -1, fx.IDX_EINVAL),
        (a["rot"], 63, fx.IDX_EINVAL), (a["rot"], 0, fx.IDX_EINVAL), (a["rot"], 514, fx.IDX_EINVAL),
        (a["offset"], 449, fx.IDX_EINVAL), (a["offset"], -1, fx.IDX_EINVAL), (a["layout"], 2, fx.IDX_EUNSUPPORTED),
        (a["mscale"], NAN, fx.IDX_EINVAL), (a["mscale"], INF, fx.IDX_EINVAL),
        (paged, (None, FAKE, 0, 100, 4), fx.IDX_EINVAL), (paged, (None, FAKE, 16, 6, 4), fx.IDX_EINVAL),
        (paged, (None, FAKE, 16, 7, 0), fx.IDX_EINVAL), (paged, (None, FAKE, 16, 7, 3), fx.IDX_EINVAL),
        ((*paged, a["ring"]), (None, FAKE, 16, 1, 4, 17), fx.IDX_EINVAL),
        (a["x"], FAKE + 1, fx.IDX_EALIGN), ((a["x"], a["dtype"]), (FAKE + 2, 1), fx.IDX_EALIGN),
        (a["codes"], FAKE + 2, fx.IDX_EALIGN), ((a["codes"], a["format"]), (FAKE + 4, 1), fx.IDX_EALIGN),
        (a["at"], FAKE + 4, fx.IDX_EALIGN), (a["base"], FAKE + 4, fx.IDX_EALIGN), (a["seq"], FAKE + 2, fx.IDX_EALIGN),
        (a["pos"], FAKE + 4, fx.IDX_EALIGN), (a["freq"], FAKE + 4, fx.IDX_EALIGN)])


def test_refusals_of_one_call(fx):
    refuse(fx, "idx_write_rows", WRITE, [
        (W["eps"], 0.0, fx.IDX_EINVAL), (W["eps"], NAN, fx.IDX_EINVAL), (W["eps"], -1.0, fx.IDX_EINVAL),
        ((W["format"], W["offset"], W["signs"]), (2, 64, None), fx.IDX_EINVAL),
        ((W["format"], W["offset"], W["signs"]), (2, 64, FAKE + 1), fx.IDX_EALIGN),
        ((W["format"], W["rot"], W["offset"]), (2, 130, 0), fx.IDX_EINVAL),
        (W["codes"], FAKE + 8, fx.IDX_EALIGN), (W["gamma"], FAKE + 2, fx.IDX_EALIGN)])
    refuse(fx, "idx_read_rows", READ, [(R["stride"], 511, fx.IDX_EINVAL), ((R["format"], R["offset"]), (2, 64), fx.IDX_EINVAL)])


def test_binding_refuses_on_the_host(fx):
    """shapes and types, before any address is used"""
    codes, scales = torch.zeros(10, 512, dtype=torch.uint8), torch.zeros(10, 16, dtype=torch.uint8)
    x, at = torch.zeros(3, 512, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int64)
    good = dict(format="local", x=x, codes=codes, scales=scales, at=at, max_n=10)
    for change, error in [
            (dict(format="fp8"), ValueError), (dict(x=x.half()), TypeError), (dict(x=x[:2]), ValueError),
            (dict(x=x[:, :500]), ValueError), (dict(x=x.t().contiguous().t()), ValueError), (dict(at=at.int()), TypeError),
            (dict(codes=codes[:, :500]), ValueError), (dict(scales=scales[:9]), ValueError),
            (dict(codes=codes.char()), TypeError), (dict(kv_base=at[:2]), ValueError),
            (dict(pages=torch.zeros(1, 2, dtype=torch.int32), page_size=4, seq=at.int()), ValueError),
            (dict(pages=torch.zeros(1, 0, dtype=torch.int32), page_size=4, seq=at.int(), max_n=0), ValueError),
            (dict(freq=torch.zeros(32, dtype=torch.float64), layout="pairs"), ValueError),
            (dict(freq=torch.zeros(32)), TypeError), (dict(eps=1e-6, gamma=torch.ones(128)), ValueError),
            (dict(gamma=torch.ones(512)), ValueError),  # without eps there is no norm for it
            (dict(), ValueError)]:  # the last: not on a GPU
        with pytest.raises(error):
            fx.idx_write_rows(**{**good, **change})
    with pytest.raises(ValueError):
        fx.idx_read_rows("local", codes, scales, at, 10, out=torch.zeros(3, 512).expand(3, 512)[:, :1].expand(3, 512))


def test_the_reference_against_the_formats():
    """E4M3 by torch's conversion (its ties go to the even code), the codes' nearness by trying every code"""
    rng = np.random.default_rng(0)
    v = np.concatenate([rng.standard_normal(4000) * 40, (ref.E4M3[1:] + ref.E4M3[:-1]) / 2, ref.E4M3]).astype(np.float32)
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(ref.E4M3[ref.nearest(v.astype(np.float64), ref.E4M3)] * np.sign(v), want)
    for format, (dim, group, width) in ref.FORMATS.items():
        y = rng.standard_normal((50, dim)) * np.exp(rng.standard_normal((50, 1)) * 2)
        codes, scales = ref.quantise(format, y)
        got = ref.values(format, codes, scales)
        table = ref.E4M3 if format == "local" else ref.E2M1
        s = ref.attn_ref.e4m3(scales) if format == "main" else 2.0 ** (scales.astype(float) - 127)
        every = np.concatenate([-table, table])[:, None, None] * np.repeat(s, group, 1)
        assert np.array_equal(np.abs(got - y), np.abs(every - y).min(0))
        # the scale: no smaller one of its kind holds the group
        top = np.abs(y.reshape(50, -1, group)).max(2)
        most = table[-1] * s
        assert (most >= top).all()
        smaller = ref.attn_ref.e4m3(scales - 1) if format == "main" else s / 2
        at_least = (scales == 112) if format == "local" else np.zeros_like(scales, bool)
        assert ((table[-1] * smaller < top) | at_least).all()


# idx_attend_local: q, nq, heads, group, codes, scales, rows, kv_base, pages, pages_stride, nseq, page_size, seq, n_vis,
# max_n, window, ring, scale, other, other_lse, pos, freq, rot, offset, layout, mscale, out, lse, ws, ws_bytes, stream
LOCAL = [FAKE, 6, 8, 3, FAKE, FAKE, 100, FAKE, None, 0, 0, 0, None, FAKE, 100, 20, 0, 0.05, FAKE, FAKE, FAKE, FAKE, 64, 448, 1,
         1.0, FAKE, FAKE, FAKE, 16, None]
L = dict(q=0, nq=1, heads=2, group=3, codes=4, scales=5, rows=6, base=7, pages=8, pstride=9, nseq=10, psize=11, seq=12, n_vis=13,
         max_n=14, window=15, ring=16, scale=17, other=18, other_lse=19, pos=20, freq=21, rot=22, offset=23, layout=24, mscale=25,
         out=26, lse=27, ws=28, ws_bytes=29)


def test_local_attention_refusals(fx):
    name, a = "idx_attend_local", L
    none = list(LOCAL)
    none[a["nq"]] = 0
    for x in ("q", "codes", "n_vis", "out", "ws", "base"):
        none[a[x]] = None
    assert call(fx, name, *none)[0] == fx.IDX_OK
    paged = (a["base"], a["pages"], a["psize"], a["pstride"], a["nseq"])
    refuse(fx, name, LOCAL, [(a[x], None, fx.IDX_EINVAL) for x in
                             ("q", "codes", "scales", "n_vis", "out", "other", "other_lse", "pos", "base")])
    refuse(fx, name, LOCAL, [
        (a["pages"], FAKE, fx.IDX_EINVAL), (a["nq"], -1, fx.IDX_EUNSUPPORTED), (a["nq"], 65538, fx.IDX_EUNSUPPORTED),
        (a["heads"], 0, fx.IDX_EUNSUPPORTED), (a["heads"], 129, fx.IDX_EUNSUPPORTED), (a["group"], 0, fx.IDX_EINVAL),
        (a["group"], 4, fx.IDX_EINVAL), (a["group"], -3, fx.IDX_EINVAL), (a["rows"], -1, fx.IDX_EUNSUPPORTED),
        (a["rows"], 1 << 31, fx.IDX_EUNSUPPORTED),
        (a["max_n"], -1, fx.IDX_EUNSUPPORTED), (a["max_n"], (1 << 30) + 1, fx.IDX_EUNSUPPORTED),
        (a["window"], -1, fx.IDX_EINVAL), (a["ring"], -1, fx.IDX_EUNSUPPORTED), (a["ring"], 21, fx.IDX_EINVAL),
        ((a["ring"], a["window"]), (22, 0), fx.IDX_EINVAL), ((a["ring"], a["window"]), (22, 1 << 62), fx.IDX_EINVAL),
        (a["scale"], NAN, fx.IDX_EINVAL), (a["scale"], INF, fx.IDX_EINVAL),
        (paged, (None, FAKE, 0, 100, 2), fx.IDX_EINVAL), (paged, (None, FAKE, 16, 6, 2), fx.IDX_EINVAL),
        (paged, (None, FAKE, 16, 7, 1), fx.IDX_EINVAL), ((*paged, a["ring"]), (None, FAKE, 11, 1, 2, 22), fx.IDX_EINVAL),
        (a["rot"], 63, fx.IDX_EINVAL), (a["rot"], 514, fx.IDX_EINVAL), (a["offset"], 449, fx.IDX_EINVAL),
        (a["layout"], 2, fx.IDX_EUNSUPPORTED), (a["mscale"], NAN, fx.IDX_EINVAL),
        (a["ws"], None, fx.IDX_EWORKSPACE), (a["ws_bytes"], 15, fx.IDX_EWORKSPACE),
        (a["q"], FAKE + 8, fx.IDX_EALIGN), (a["codes"], FAKE + 8, fx.IDX_EALIGN), (a["scales"], FAKE + 2, fx.IDX_EALIGN),
        (a["n_vis"], FAKE + 2, fx.IDX_EALIGN), (a["other"], FAKE + 8, fx.IDX_EALIGN), (a["other_lse"], FAKE + 2, fx.IDX_EALIGN),
        (a["out"], FAKE + 8, fx.IDX_EALIGN), (a["lse"], FAKE + 2, fx.IDX_EALIGN), (a["ws"], FAKE + 8, fx.IDX_EALIGN),
        (a["base"], FAKE + 4, fx.IDX_EALIGN), (a["seq"], FAKE + 2, fx.IDX_EALIGN), (a["pos"], FAKE + 4, fx.IDX_EALIGN),
        (a["freq"], FAKE + 4, fx.IDX_EALIGN)])


def test_local_workspace_sizes(fx):
    op = fx.IDX_OP_ATTEND_LOCAL
    assert fx.workspace_size(op, 4096, 128, 64) == 16
    assert fx.workspace_size(op, 1, 1 << 30, 128) > 16
    assert fx.workspace_size(op, 0, 100, 1) == 16 and fx.workspace_size(op, 5, 0, 1) == 16
    assert fx.workspace_size(op, 5, 100, 129) == 0 and fx.workspace_size(op, -1, 100, 1) == 0


def test_local_attention_binding_refuses_on_the_host(fx):
    q, codes = torch.zeros(4, 2, 512, dtype=torch.bfloat16), torch.zeros(10, 512, dtype=torch.uint8)
    good = dict(q=q, codes=codes, scales=torch.zeros(10, 16, dtype=torch.uint8), n_vis=torch.zeros(4, dtype=torch.int32), max_n=10,
                scale=1.0, out=q.clone(), ws=torch.zeros(16, dtype=torch.uint8), group=2, kv_base=torch.zeros(2, dtype=torch.int64))
    for change, error in [
            (dict(q=q[..., :256]), ValueError), (dict(q=q.float()), TypeError), (dict(group=3), ValueError),
            (dict(group=0), ValueError), (dict(n_vis=good["n_vis"][:2]), ValueError), (dict(codes=codes[:9]), ValueError),
            (dict(kv_base=torch.zeros(4, dtype=torch.int64)), ValueError), (dict(out=q[:, :1]), ValueError),
            (dict(other=q.float(), other_lse=torch.zeros(4, 2)), TypeError),
            (dict(other=q, other_lse=torch.zeros(4)), ValueError), (dict(lse=torch.zeros(2, 4)), ValueError),
            (dict(freq=torch.zeros(32, dtype=torch.float64), pos=torch.zeros(2, dtype=torch.int64)), ValueError),
            (dict(), ValueError)]:  # the last: not on a GPU
        with pytest.raises(error):
            fx.idx_attend_local(**{**good, **change})
