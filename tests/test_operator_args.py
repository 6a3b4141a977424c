"""Argument checks of the rotary, attention and distillation entry points, before any HIP call (no GPU), and
the frequencies of idx_rope_freqs against their formulas."""
import ctypes
import math

import numpy as np
import pytest
import torch

from test_abi import FAKE, call, fx  # noqa: F401

NAN, INF = math.nan, math.inf


def refuse(fx, name, good, cases):
    for i, v, st in cases:
        bad = list(good)
        for j, x in zip(i, v) if isinstance(i, tuple) else [(i, v)]:
            bad[j] = x
        got, msg = call(fx, name, *bad)
        assert got == st, (name, i, v, got, msg)
        assert name in msg


def test_rope_refusals(fx):
    # x, dtype, tokens, heads, dim, x_token, x_head, pos, freq, rot, offset, layout, mscale, inverse, out, out_token,
    # out_head, stream
    good = [FAKE, 0, 4, 2, 128, 256, 128, FAKE, FAKE, 64, 64, 0, 1.0, 0, FAKE + 4096, 256, 128, None]
    none = list(good); none[2] = 0; none[0] = none[14] = None
    assert call(fx, "idx_rope", *none)[0] == fx.IDX_OK
    refuse(fx, "idx_rope", good, [
        (0, None, fx.IDX_EINVAL), (7, None, fx.IDX_EINVAL), (8, None, fx.IDX_EINVAL), (14, None, fx.IDX_EINVAL),
        (1, 2, fx.IDX_EUNSUPPORTED), (11, 2, fx.IDX_EUNSUPPORTED), (2, -1, fx.IDX_EUNSUPPORTED),
        (2, 1 << 31, fx.IDX_EUNSUPPORTED), (3, 0, fx.IDX_EUNSUPPORTED), (3, 65536, fx.IDX_EUNSUPPORTED),
        (4, 1, fx.IDX_EUNSUPPORTED), (4, (1 << 20) + 2, fx.IDX_EUNSUPPORTED),
        (9, 63, fx.IDX_EINVAL), (9, 0, fx.IDX_EINVAL), (9, 130, fx.IDX_EINVAL), (9, -2, fx.IDX_EINVAL),
        ((4, 9, 10, 15, 16, 5, 6), (16384, 8194, 0, 32768, 16384, 32768, 16384), fx.IDX_EINVAL),
        (10, 65, fx.IDX_EINVAL), (10, -1, fx.IDX_EINVAL), (12, NAN, fx.IDX_EINVAL), (12, INF, fx.IDX_EINVAL),
        (5, -1, fx.IDX_EINVAL), (6, -1, fx.IDX_EINVAL), (15, 127, fx.IDX_EINVAL), (16, 0, fx.IDX_EINVAL),
        ((14, 15), (FAKE, 512), fx.IDX_EINVAL),  # in place with other strides
        (0, FAKE + 1, fx.IDX_EALIGN), (14, FAKE + 4097, fx.IDX_EALIGN), (7, FAKE + 4, fx.IDX_EALIGN),
        (8, FAKE + 4, fx.IDX_EALIGN), ((0, 1), (FAKE + 2, 1), fx.IDX_EALIGN)])


def test_rope_outputs_that_overlap(fx):
    """rows dim apart are not enough: the heads of a token must end before the next token's, or the other way round"""
    at = dict(tokens=2, heads=3, out_token=15, out_head=16)
    good = [FAKE, 0, 4, 2, 128, 256, 128, FAKE, FAKE, 64, 64, 0, 1.0, 0, FAKE + 4096, 256, 128, None]
    refuse(fx, "idx_rope", good, [
        ((at["out_token"], at["out_head"]), v, fx.IDX_EINVAL)
        for v in ((128, 128), (255, 128), (128, 511), (129, 500), (200, 300))])
    refuse(fx, "idx_rope", good, [(at["tokens"], 1 << 24, fx.IDX_EUNSUPPORTED)])


ATTEND = dict(q=0, nq=1, heads=2, codes=3, scales=4, rows=5, base=6, pages=7, pstride=8, nseq=9, psize=10, seq=11, nvis=12,
              maxn=13)


def common_refusals(fx, name, good, at):
    """`at`: names of the arguments that both attention calls have -> places"""
    a = at
    refuse(fx, name, good, [
        (a["q"], None, fx.IDX_EINVAL), (a["codes"], None, fx.IDX_EINVAL), (a["scales"], None, fx.IDX_EINVAL),
        (a["nvis"], None, fx.IDX_EINVAL), (a["base"], None, fx.IDX_EINVAL),
        (a["pages"], FAKE, fx.IDX_EINVAL),  # both forms at once
        (a["nq"], -1, fx.IDX_EUNSUPPORTED), (a["nq"], 65536, fx.IDX_EUNSUPPORTED), (a["heads"], 0, fx.IDX_EUNSUPPORTED),
        (a["heads"], 129, fx.IDX_EUNSUPPORTED), (a["rows"], -1, fx.IDX_EUNSUPPORTED),
        (a["rows"], 1 << 31, fx.IDX_EUNSUPPORTED), (a["maxn"], -1, fx.IDX_EUNSUPPORTED),
        (a["maxn"], (1 << 30) + 1, fx.IDX_EUNSUPPORTED), (a["scale"], NAN, fx.IDX_EINVAL), (a["scale"], INF, fx.IDX_EINVAL),
        ((a["base"], a["pages"], a["psize"]), (None, FAKE, 0), fx.IDX_EINVAL),
        ((a["base"], a["pages"], a["psize"], a["pstride"]), (None, FAKE, 16, 6), fx.IDX_EINVAL),
        ((a["base"], a["pages"], a["psize"], a["pstride"]), (None, FAKE, 16, 7), fx.IDX_EINVAL),  # nseq 0
        ((a["base"], a["pages"], a["psize"], a["pstride"], a["nseq"]), (None, FAKE, 16, 7, 3), fx.IDX_EINVAL),
        ((a["idx"], a["istride"]), (FAKE, 11), fx.IDX_EINVAL), ((a["idx"], a["k"]), (FAKE, -1), fx.IDX_EUNSUPPORTED),
        ((a["idx"], a["k"], a["istride"]), (FAKE, (1 << 24) + 1, 1 << 25), fx.IDX_EUNSUPPORTED),
        (a["q"], FAKE + 8, fx.IDX_EALIGN), (a["codes"], FAKE + 4, fx.IDX_EALIGN), (a["scales"], FAKE + 1, fx.IDX_EALIGN),
        (a["base"], FAKE + 4, fx.IDX_EALIGN), (a["nvis"], FAKE + 2, fx.IDX_EALIGN), (a["idx"], FAKE + 2, fx.IDX_EALIGN),
        (a["seq"], FAKE + 2, fx.IDX_EALIGN)])


def test_attend_refusals(fx):
    # .., window, idx, idx_stride, k, scale, out, lse, ws, ws_bytes, stream
    ws = fx.workspace_size(fx.IDX_OP_ATTEND, 4, 100, 64)
    good = [FAKE, 4, 64, FAKE, FAKE, 1000, FAKE, None, 0, 0, 0, None, FAKE, 100, 0, None, 12, 12, 0.1, FAKE, FAKE, FAKE, ws,
            None]
    none = list(good); none[1] = 0; none[0] = none[3] = none[6] = none[12] = none[19] = none[21] = None
    assert call(fx, "idx_attend", *none)[0] == fx.IDX_OK
    common_refusals(fx, "idx_attend", good, dict(ATTEND, idx=15, istride=16, k=17, scale=18))
    refuse(fx, "idx_attend", good, [
        (14, -1, fx.IDX_EINVAL), ((14, 15), (5, FAKE), fx.IDX_EINVAL), (19, None, fx.IDX_EINVAL),
        (19, FAKE + 8, fx.IDX_EALIGN), (20, FAKE + 2, fx.IDX_EALIGN), (21, FAKE + 8, fx.IDX_EALIGN),
        (21, None, fx.IDX_EWORKSPACE), (22, ws - 1, fx.IDX_EWORKSPACE)])
    assert fx.workspace_size(fx.IDX_OP_ATTEND, 4, 100, 129) == 0
    assert fx.workspace_size(fx.IDX_OP_ATTEND, 4, -1, 64) == 0
    # a window or a list needs no more than its own length
    assert fx.workspace_size(fx.IDX_OP_ATTEND, 1, 64, 64) < fx.workspace_size(fx.IDX_OP_ATTEND, 1, 1 << 20, 64) < 1 << 28


def test_attend_weights_refusals(fx):
    # .., idx, idx_stride, k, scale, lse, weights, w_stride, stream
    good = [FAKE, 4, 64, FAKE, FAKE, 1000, FAKE, None, 0, 0, 0, None, FAKE, 100, None, 12, 12, 0.1, FAKE, FAKE, 100, None]
    none = list(good); none[1] = 0; none[0] = none[3] = none[6] = none[12] = none[18] = none[19] = None
    assert call(fx, "idx_attend_weights", *none)[0] == fx.IDX_OK
    common_refusals(fx, "idx_attend_weights", good, dict(ATTEND, idx=14, istride=15, k=16, scale=17))
    refuse(fx, "idx_attend_weights", good, [
        (18, None, fx.IDX_EINVAL), (19, None, fx.IDX_EINVAL), (20, 99, fx.IDX_EINVAL),
        ((14, 20), (FAKE, 11), fx.IDX_EINVAL), (18, FAKE + 2, fx.IDX_EALIGN), (19, FAKE + 2, fx.IDX_EALIGN)])


def test_distill_refusals(fx):
    ws = fx.workspace_size(fx.IDX_OP_DISTILL, 4, 100000, 1)
    # scores, stride, n_vis, nq, max_n, t_idx, t_logit, t_stride, k, inv_temp | loss, lse, t_lse, ws, bytes, stream
    fwd = [FAKE, 100000, FAKE, 4, 100000, FAKE, FAKE, 64, 64, 1.0, FAKE, FAKE, FAKE, FAKE, ws, None]
    bwd = fwd[:10] + [FAKE, FAKE, FAKE, FAKE + 4096, 100000, None]  # lse, t_lse, dloss, dscores, d_stride, stream
    shared = [(0, None, fx.IDX_EINVAL), (2, None, fx.IDX_EINVAL), (5, None, fx.IDX_EINVAL), (6, None, fx.IDX_EINVAL),
              (1, 99999, fx.IDX_EINVAL), (7, 63, fx.IDX_EINVAL), (8, -1, fx.IDX_EUNSUPPORTED),
              ((7, 8), (4096, 2049), fx.IDX_EUNSUPPORTED), (3, -1, fx.IDX_EUNSUPPORTED), (3, 65536, fx.IDX_EUNSUPPORTED),
              (4, -1, fx.IDX_EUNSUPPORTED), ((1, 4), (1 << 31, (1 << 30) + 1), fx.IDX_EUNSUPPORTED),
              (9, 0.0, fx.IDX_EINVAL), (9, -1.0, fx.IDX_EINVAL), (9, NAN, fx.IDX_EINVAL), (9, INF, fx.IDX_EINVAL),
              (0, FAKE + 2, fx.IDX_EALIGN), (2, FAKE + 2, fx.IDX_EALIGN), (5, FAKE + 2, fx.IDX_EALIGN),
              (6, FAKE + 2, fx.IDX_EALIGN), (10, None, fx.IDX_EINVAL), (11, None, fx.IDX_EINVAL),
              (12, None, fx.IDX_EINVAL), (10, FAKE + 2, fx.IDX_EALIGN), (11, FAKE + 2, fx.IDX_EALIGN),
              (12, FAKE + 2, fx.IDX_EALIGN)]
    refuse(fx, "idx_distill", fwd, shared + [(13, None, fx.IDX_EWORKSPACE), (14, ws - 1, fx.IDX_EWORKSPACE),
                                             (13, FAKE + 8, fx.IDX_EALIGN)])
    refuse(fx, "idx_distill_bwd", bwd, shared + [(13, None, fx.IDX_EINVAL), (14, 99999, fx.IDX_EINVAL),
                                                 (13, FAKE + 4098, fx.IDX_EALIGN),
                                                 ((13, 14), (FAKE, 100004), fx.IDX_EINVAL)])
    for name, good in (("idx_distill", fwd), ("idx_distill_bwd", bwd)):
        none = list(good); none[3] = 0; none[0] = none[2] = none[5] = None
        assert call(fx, name, *none)[0] == fx.IDX_OK


def test_rope_frequencies(fx):
    """the fp64 formulas, evaluated here with another power function: a few units of 2^-53 each"""
    rot, base, factor, original = 64, 10000.0, 8.0, 4096.0
    f = np.array([math.exp(-2.0 * i / rot * math.log(base)) for i in range(rot // 2)])
    ntk = np.array([math.exp(-2.0 * i / rot * (math.log(base) + rot / (rot - 2) * math.log(factor))) for i in range(rot // 2)])
    turns = original * f / (2 * math.pi)
    keep = np.clip((turns - 1.0) / 31.0, 0, 1)
    want = dict(plain=f, linear=f / factor, ntk=ntk, yarn=f * keep + f / factor * (1 - keep))
    for scaling, w in want.items():
        got, ms = fx.rope_freqs(rot, base, scaling, factor, original, device="cpu")
        assert got.dtype == torch.float64 and (np.abs(got.numpy() / w - 1) < 1e-13).all(), scaling
        assert ms == (np.float32(0.1 * math.log(8.0) + 1) if scaling == "yarn" else 1.0)
    assert want["yarn"][0] == f[0] and abs(want["yarn"][-1] / (f[-1] / factor) - 1) < 1e-15  # both ends of the ramp
    assert (keep > 0).sum() > (keep == 1).sum() > 0
    buf, ms = (ctypes.c_double * 4096)(), ctypes.c_float()
    good = [64, 10000.0, 3, 8.0, 4096.0, 32.0, 1.0, ctypes.addressof(buf), ctypes.addressof(ms)]
    refuse(fx, "idx_rope_freqs", good, [
        (0, 0, fx.IDX_EINVAL), (0, 7, fx.IDX_EINVAL), (0, 8194, fx.IDX_EINVAL), (1, 1.0, fx.IDX_EINVAL),
        (1, NAN, fx.IDX_EINVAL), (1, INF, fx.IDX_EINVAL), (2, 4, fx.IDX_EUNSUPPORTED), (2, -1, fx.IDX_EUNSUPPORTED),
        (3, 0.5, fx.IDX_EINVAL), (3, INF, fx.IDX_EINVAL), (4, 0.0, fx.IDX_EINVAL), (5, 1.0, fx.IDX_EINVAL),
        (6, NAN, fx.IDX_EINVAL), (7, None, fx.IDX_EINVAL), (8, None, fx.IDX_EINVAL),
        ((0, 2), (2, 2), fx.IDX_EINVAL)])
    with pytest.raises(ValueError):
        fx.rope_freqs(64, scaling="other")


def test_python_calls_refuse_what_they_cannot_take(fx):
    """types, shapes and places, before the library is called (CPU tensors: no GPU here)"""
    b, f, i = torch.bfloat16, torch.float32, torch.int32
    freq = fx.rope_freqs(64, device="cpu")[0]
    pos = torch.zeros(4, dtype=torch.int64)
    x = torch.zeros(4, 2, 128, dtype=b)
    for bad, err in ((dict(x=x.half()), TypeError), (dict(x=x[0]), ValueError), (dict(x=x.transpose(1, 2)), ValueError),
                     (dict(pos=pos.int()), TypeError), (dict(pos=pos[:3]), ValueError), (dict(freq=freq.float()), TypeError),
                     (dict(layout="other"), ValueError), (dict(out=x.float()), TypeError),
                     (dict(out=torch.zeros(4, 2, 64, dtype=b)), ValueError)):
        with pytest.raises(err):
            fx.idx_rope(**dict(dict(x=x, pos=pos, freq=freq), **bad))
    q = torch.zeros(3, 8, 512, dtype=b)
    args = dict(q=q, codes=torch.zeros(9, 256, dtype=torch.uint8), scales=torch.zeros(9, 32, dtype=torch.uint8),
                n_vis=torch.zeros(3, dtype=i), max_n=9, scale=1.0, kv_base=torch.zeros(3, dtype=torch.int64))
    out, ws = torch.zeros_like(q), torch.zeros(1 << 20, dtype=torch.uint8)
    lse, w = torch.zeros(3, 8), torch.zeros(3, 9)
    for bad, err in ((dict(q=q.float()), TypeError), (dict(codes=args["codes"].char()), TypeError),
                     (dict(scales=args["scales"][:8]), ValueError), (dict(n_vis=args["n_vis"][:2]), ValueError),
                     (dict(kv_base=args["kv_base"].int()), TypeError), (dict(kv_base=args["kv_base"][:2]), ValueError),
                     (dict(seq=torch.zeros(3)), TypeError), (dict(idx=torch.zeros(3, 4)), TypeError)):
        with pytest.raises(err):
            fx.idx_attend(**dict(args, out=out, ws=ws, **bad) if not set(bad) & set(args) else dict(args, **bad, out=out, ws=ws))
        with pytest.raises(err):
            fx.idx_attend_weights(**dict(args, lse=lse, weights=w, **bad) if not set(bad) & set(args) else
                                  dict(args, **bad, lse=lse, weights=w))
    for bad, err in ((dict(out=out.float()), TypeError), (dict(out=out[:2]), ValueError), (dict(lse=lse[:, :7]), ValueError),
                     (dict(), ValueError)):  # CPU tensors
        with pytest.raises(err):
            fx.idx_attend(**{**args, "out": out, "ws": ws, **bad})
    s, ti, tl, r = torch.zeros(3, 9), torch.zeros(3, 4, dtype=i), torch.zeros(3, 4), torch.zeros(3)
    good = dict(scores=s, n_vis=args["n_vis"], max_n=9, t_idx=ti, t_logit=tl, loss=r, lse=r, t_lse=r, ws=ws)
    for bad, err in ((dict(scores=s.bfloat16()), TypeError), (dict(scores=s[:2]), ValueError), (dict(t_idx=ti.long()), TypeError),
                     (dict(t_logit=tl[:, :3]), ValueError), (dict(loss=r[:2]), ValueError), (dict(lse=r.double()), TypeError),
                     (dict(), ValueError)):
        with pytest.raises(err):
            fx.idx_distill(**{**good, **bad})
