"""idx_write_rows and idx_read_rows against their 64-bit definitions (rows_ref.py). Codes and scales are compared exactly:
both sides decide in 64 bits, and no drawn value lies within their error (2^-45 of it) of a border unless it lies on it."""
import itertools

import numpy as np
import pytest
import torch

import rows_ref as ref

pytestmark = pytest.mark.gpu
FILL = 0xA5


@pytest.fixture(scope="module")
def fx():
    import top_fp4_lightning_amd as fx

    return fx


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


def bf16(x):
    """nearest bf16 of fp32 values, as fp32"""
    return torch.from_numpy(np.asarray(x, np.float32)).bfloat16().float().numpy()


def places(kind, rng, tokens, rows):
    """Arguments that say where entries lie, and the entries: distinct rows, with some that are not there"""
    seqs = 3
    if kind == "rows":  # entries are cache rows
        at = rng.permutation(rows)[:tokens].astype(np.int64)
        w = dict(max_n=rows)
    elif kind == "base":
        at = rng.integers(0, 20, tokens)
        base = rng.permutation(rows)[:tokens] - at
        w = dict(max_n=21, kv_base=base.astype(np.int64))
    else:
        page, ring = 7, 52 if kind == "ring" else 0
        per = -(-ring // page) if ring else rows // page // seqs
        pages = rng.permutation(rows // page)[:seqs * per].reshape(seqs, per).astype(np.int32)
        seq = (np.arange(tokens) % seqs).astype(np.int32)
        first = 1000 if ring else 3
        at = first + np.arange(tokens) // seqs
        w = dict(max_n=10_000 if ring else per * page, pages=pages, page_size=page, seq=seq, ring=ring)
        if tokens > 20:
            pages[1, 1] = -1  # a page that is not there
            pages[2, 2] = rows // page + 5  # and one past the cache
            seq[4], seq[8] = -1, seqs
    if tokens > 20:
        at[2], at[11] = -1, w["max_n"]
    return {k: (dev(v) if isinstance(v, np.ndarray) else v) for k, v in w.items()}, at, \
        {k: v for k, v in w.items() if k != "max_n"}, w["max_n"]


TURNS = [None, dict(rot=64, offset="last", layout="interleaved", mscale=1.0), dict(rot=34, offset=5, layout="interleaved", mscale=1.25),
         dict(rot=64, offset="last", layout="half", mscale=1.5), dict(rot=102, offset=3, layout="half", mscale=1.0),
         dict(rot="dim", offset=0, layout="half", mscale=1.0), dict(rot="dim", offset=0, layout="interleaved", mscale=0.5)]


def turn_of(i, dim, tokens, rng, far=1 << 20):
    t = TURNS[i]
    if t is None:
        return {}, None
    rot = dim if t["rot"] == "dim" else t["rot"]
    offset = dim - rot if t["offset"] == "last" else t["offset"]
    freq = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    pos = rng.integers(0, far, tokens)
    return dict(pos=dev(pos), freq=dev(freq), offset=offset, layout=t["layout"], mscale=t["mscale"]), \
        (pos, freq, offset, t["layout"], t["mscale"])


def wanted(format, x, gamma, eps, turn, signs):
    y = np.asarray(x, np.float64)
    if eps is not None:
        y = ref.normalise(y, gamma, eps)
    if turn is not None:
        y = ref.rotate(y, *turn)
    if format == "key":
        y = ref.transform(y, signs)
    return ref.quantise(format, y)


@pytest.mark.parametrize("format", ["main", "local", "key"])
@pytest.mark.parametrize("i, kind, tokens", [(i, k, n) for i, (k, n) in enumerate(
    itertools.product(["rows", "base", "pages", "ring"], [1, 6, 150]))])
def test_write(fx, format, i, kind, tokens):
    dim, group, width = ref.FORMATS[format]
    rng = np.random.default_rng(100 * i + len(format))
    rows = 1001
    w, at, where, max_n = places(kind, rng, tokens, rows)
    f32, norm, pad = bool(i & 1), (i // 2) % 3, (0, 64, 7)[i % 3]
    x = rng.standard_normal((tokens, dim + pad)) * np.exp(rng.standard_normal((tokens, 1)) * 2)
    x = np.float32(x) if f32 else bf16(x)
    gamma = np.float32(1 + 0.3 * rng.standard_normal(dim)) if norm == 2 else None
    eps = 1e-5 if norm else None
    kw, turn = turn_of(i % len(TURNS), dim, tokens, rng)
    signs = rng.integers(0, 2, 128).astype(np.int8) * 2 - 1
    want_codes, want_scales = wanted(format, x[:, pad:], gamma, eps, turn, signs)
    codes = torch.full((rows, width), FILL, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, dim // group), FILL, dtype=torch.uint8, device="cuda")
    fx.idx_write_rows(format, dev(x, torch.float32 if f32 else torch.bfloat16)[:, pad:], codes, scales, dev(at),
                      gamma=None if gamma is None else dev(gamma), eps=eps, signs=dev(signs), **w, **kw)
    all_codes, all_scales = np.full((rows, width), FILL, np.uint8), np.full((rows, dim // group), FILL, np.uint8)
    for t in range(tokens):
        r = ref.row_of(t, at, max_n, rows, **where)
        if r >= 0:
            all_codes[r], all_scales[r] = want_codes[t], want_scales[t]
    assert (all_codes != FILL).any()
    assert np.array_equal(scales.cpu().numpy(), all_scales)
    assert np.array_equal(codes.cpu().numpy(), all_codes)


@pytest.mark.parametrize("format", ["main", "local", "key"])
def test_write_borders(fx, format):
    """values on and next to every border, zeros of both signs, groups of zeros, tiny and huge groups"""
    dim, group, width = ref.FORMATS[format]
    rng = np.random.default_rng(1)
    table = ref.E4M3 if format == "local" else ref.E2M1
    mid = (table[1:] + table[:-1]) / 2
    edge = np.concatenate([mid, table, mid * (1 + 2.0 ** -22), mid * (1 - 2.0 ** -22)])
    v = np.zeros((40, dim))
    for r in range(40):
        v[r] = rng.choice(edge, dim) * rng.choice([-1, 1], dim)
        v[r, ::group] = table[-1]  # the scale below
        s = 2.0 ** float(rng.integers(-14, 7)) if format != "main" else rng.choice(ref.E4M3[1:])
        v[r] *= s
    v[20, :group] = 0.0
    v[21, 3 * group:] = -0.0
    v[22] *= 2.0 ** -30
    v[23] *= 2.0 ** 20
    v[24] = 3e38
    v[25] = 1e-42
    v[26] = rng.standard_normal(dim) * 2.0 ** -20
    v[27, 0::2], v[27, 1::2] = 1.0, -2.0 ** -26
    x = np.float32(v)
    if format == "key":  # the transform of the transform is 128 / sqrt(128)^2 times the row
        x = x[:24]
    signs = np.ones(128, np.int8)
    codes = torch.zeros(len(x), width, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(len(x), dim // group, dtype=torch.uint8, device="cuda")
    at = torch.arange(len(x), device="cuda")
    fx.idx_write_rows(format, dev(x), codes, scales, at, len(x), signs=dev(signs))
    want = wanted(format, x, None, None, None, signs)
    assert np.array_equal(scales.cpu().numpy(), want[1])
    assert np.array_equal(codes.cpu().numpy(), want[0])
    # turned by no angle: the same through the 64-bit path
    again = torch.zeros_like(codes)
    scales.zero_()
    fx.idx_write_rows(format, dev(x), again, scales, at, len(x), signs=dev(signs), pos=torch.zeros_like(at),
                      freq=torch.ones(dim // 2, dtype=torch.float64, device="cuda"), layout="interleaved")
    assert torch.equal(again, codes)
    assert np.array_equal(scales.cpu().numpy(), want[1])


def test_write_as_the_codecs(fx):
    """plain bf16 rows: what idx_quantize_kv and idx_quantize_q store"""
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(333, 512, device="cuda", generator=g).bfloat16()
    codes, scales = fx.idx_quantize_kv(x)
    at = torch.randperm(400, device="cuda", generator=g)[:333]
    c, s = torch.zeros(400, 256, dtype=torch.uint8, device="cuda"), torch.zeros(400, 32, dtype=torch.uint8, device="cuda")
    fx.idx_write_rows("main", x, c, s, at, 400)
    assert torch.equal(c[at], codes) and torch.equal(s[at], scales)
    k = torch.randn(333, 128, device="cuda", generator=g).bfloat16()
    signs = (torch.randint(0, 2, (128,), device="cuda", generator=g) * 2 - 1).to(torch.int8)
    codes, scales = fx.idx_quantize_q(k, signs)
    c, s = torch.zeros(400, 64, dtype=torch.uint8, device="cuda"), torch.zeros(400, 4, dtype=torch.uint8, device="cuda")
    fx.idx_write_rows("key", k, c, s, at, 400, signs=signs)
    assert torch.equal(c[at], codes) and torch.equal(s[at], scales)


@pytest.mark.parametrize("format", ["main", "local", "key"])
@pytest.mark.parametrize("i, kind, tokens", [(i, k, n) for i, (k, n) in enumerate(
    itertools.product(["rows", "base", "pages", "ring"], [1, 70]))])
def test_read(fx, format, i, kind, tokens):
    """every byte that is a number; entries that are not there are zeros, and what lies in their rows has no effect"""
    dim, group, width = ref.FORMATS[format]
    rng = np.random.default_rng(7 * i + len(format))
    rows = 515
    w, at, where, max_n = places(kind, rng, tokens, rows)
    codes = rng.integers(0, 256, (rows, width)).astype(np.uint8)
    if format == "local":
        codes[(codes & 127) == 127] = 0
        scales = rng.integers(112, 135, (rows, 16)).astype(np.uint8)
    elif format == "main":
        scales = rng.integers(0, 256, (rows, 32)).astype(np.uint8)
        scales[(scales & 127) == 127] = 1
    else:
        scales = rng.integers(100, 150, (rows, 4)).astype(np.uint8)
    kw, turn = ({}, None) if format == "key" else turn_of(i % len(TURNS), dim, tokens, rng)
    inverse = bool(i & 2)
    exact = np.zeros((tokens, dim))
    seen = [ref.row_of(t, at, max_n, rows, **where) for t in range(tokens)]
    for t, r in enumerate(seen):
        if r >= 0:
            exact[t] = ref.values(format, codes[r:r + 1], scales[r:r + 1])[0]
    bad = np.ones(rows, bool)
    bad[[r for r in seen if r >= 0]] = False
    codes[bad] = 0xFF
    size = np.abs(exact)
    if turn is not None:
        pos, freq, offset, layout, m = turn
        exact = ref.rotate(exact, *turn, inverse=inverse)
        # of |x0 cos| + |x1 sin| <= |x0| + |x1|: the angle 2^-23 rad and its halves' rounding 2^-22, sin and cos 2^-22,
        # mscale and its product 2^-23, the two products and the sum 3 * 2^-24
        size = max(1.0, m) * (size + partner(size, freq, offset, layout))
    for dtype, eps in ((torch.float32, 0.0), (torch.bfloat16, 2.0 ** -8)):
        for pad in (0, 3):
            out = torch.full((tokens, dim + pad), 5.0, dtype=dtype, device="cuda")
            fx.idx_read_rows(format, dev(codes), dev(scales), dev(at), out=out[:, :dim], inverse=inverse, **w, **kw)
            got = out.double().cpu().numpy()
            assert (got[:, dim:] == 5.0).all()
            room = np.zeros_like(size) if turn is None else 2.0 ** -20 * size
            assert (np.abs(got[:, :dim] - exact) <= (0.0 if turn is None else eps) * np.abs(exact) * (1 + 2.0 ** -10) + room).all()


def partner(size, freq, offset, layout):
    """|other value of the pair|, 0 outside the rotated part"""
    h, y = len(freq), np.zeros_like(size)
    i0 = offset + (np.arange(h) if layout == "half" else 2 * np.arange(h))
    i1 = i0 + (h if layout == "half" else 1)
    y[:, i0], y[:, i1] = size[:, i1], size[:, i0]
    return y


def test_far_positions(fx):
    """angles of positions up to 2^31 in a format of few bits: the turned value against extended precision"""
    rng = np.random.default_rng(5)
    pos = np.array([2 ** 31, 2 ** 31 - 1, 2 ** 30 + 12345, 1 << 24, 7], np.int64)
    freq = 10000.0 ** (-np.arange(0, 64, 2) / 64)
    x = bf16(rng.standard_normal((5, 512)))
    two_pi = np.longdouble("6.283185307179586476925286766559005768")
    a = np.longdouble(pos)[:, None] * np.longdouble(freq)
    a = np.float64(a - np.rint(a / two_pi) * two_pi)
    y = x.astype(np.float64)
    c, s = np.cos(a), np.sin(a)
    y[:, 448:480], y[:, 480:] = x[:, 448:480] * c - x[:, 480:] * s, x[:, 480:] * c + x[:, 448:480] * s
    for format in ("main", "local"):
        want = ref.quantise(format, y)
        dim, group, width = ref.FORMATS[format]
        codes = torch.zeros(5, width, dtype=torch.uint8, device="cuda")
        scales = torch.zeros(5, dim // group, dtype=torch.uint8, device="cuda")
        fx.idx_write_rows(format, dev(x, torch.bfloat16), codes, scales, torch.arange(5, device="cuda"), 5, pos=dev(pos),
                          freq=dev(freq))
        assert np.array_equal(codes.cpu().numpy(), want[0]) and np.array_equal(scales.cpu().numpy(), want[1])


def test_rows_past_32_bits(fx):
    """a cache of more than 2^32 bytes"""
    rows = (1 << 23) + 100
    codes = torch.zeros(rows, 512, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(rows, 16, dtype=torch.uint8, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(4, 512, device="cuda", generator=g).bfloat16()
    at = torch.tensor([0, 5, 6, 7], device="cuda")
    base = torch.tensor([rows - 1, rows - 60, 3, -7], device="cuda")
    fx.idx_write_rows("local", x, codes, scales, at, 8, kv_base=base)
    small_c, small_s = torch.zeros(4, 512, dtype=torch.uint8, device="cuda"), torch.zeros(4, 16, dtype=torch.uint8, device="cuda")
    fx.idx_write_rows("local", x, small_c, small_s, torch.arange(4, device="cuda"), 4)
    where = at + base
    assert torch.equal(codes[where], small_c) and torch.equal(scales[where], small_s)
    assert int((codes != 0).any(1).sum()) == 4
    got = fx.idx_read_rows("local", codes, scales, at, 8, kv_base=base)
    assert torch.equal(got, fx.idx_read_rows("local", small_c, small_s, torch.arange(4, device="cuda"), 4))


def test_the_most_tokens(fx):
    """2^24 - 1 of them, one row of x for all: the first and the last have a place"""
    tokens = (1 << 24) - 1
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(1, 128, device="cuda", generator=g).bfloat16()
    signs = torch.ones(128, dtype=torch.int8, device="cuda")
    at = torch.full((tokens,), -1, dtype=torch.int64, device="cuda")
    at[0], at[-1] = 3, 1
    codes, scales = torch.zeros(5, 64, dtype=torch.uint8, device="cuda"), torch.zeros(5, 4, dtype=torch.uint8, device="cuda")
    fx.idx_write_rows("key", x.expand(tokens, 128), codes, scales, at, 5, signs=signs, kv_base=torch.zeros_like(at))
    want = fx.idx_quantize_q(x, signs)
    for row in (1, 3):
        assert torch.equal(codes[row], want[0][0]) and torch.equal(scales[row], want[1][0])
    assert not codes[[0, 2, 4]].any() and not scales[[0, 2, 4]].any()
    out = fx.idx_read_rows("key", codes, scales, at, 5, kv_base=torch.zeros_like(at))
    few = fx.idx_read_rows("key", codes, scales, at[:1], 5, kv_base=torch.zeros_like(at[:1]))
    assert few.any() and torch.equal(out[:1], few) and torch.equal(out[-1:], few) and not out[1:-1].any()


def test_nothing_to_do(fx):
    none = torch.zeros(0, 512, dtype=torch.uint8, device="cuda")
    x, at = torch.zeros(2, 512, device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda")
    fx.idx_write_rows("local", x, none, none[:, :16].contiguous(), at, 5)
    out = fx.idx_read_rows("local", none, none[:, :16].contiguous(), at, 5, dtype=torch.float32)
    assert (out == 0).all()
    c, s = torch.zeros(4, 512, dtype=torch.uint8, device="cuda"), torch.zeros(4, 16, dtype=torch.uint8, device="cuda")
    fx.idx_write_rows("local", x[:0], c, s, at[:0], 5)
    assert fx.idx_read_rows("local", c, s, at[:0], 5).shape == (0, 512)
    fx.idx_write_rows("local", x + 1, c, s, at, 0)  # no entry has a place
    assert not c.any()


def test_a_captured_step_on_another_stream(fx):
    """a ring written and read by a replayed graph: every replay with other rows and entries, eager work between"""
    g = torch.Generator(device="cuda").manual_seed(9)
    x, at = torch.empty(6, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(6, dtype=torch.int64, device="cuda")
    seq = torch.tensor([0, 1, 2, 0, 1, 2], dtype=torch.int32, device="cuda")
    pages = torch.tensor([[4, 0], [1, 3], [5, 2]], dtype=torch.int32, device="cuda")
    freq, m = fx.rope_freqs(64)
    gamma = torch.rand(512, device="cuda", generator=g) + 0.5
    caches = [(torch.zeros(60, 512, dtype=torch.uint8, device="cuda"), torch.zeros(60, 16, dtype=torch.uint8, device="cuda"))
              for _ in range(2)]
    out = torch.empty(6, 512, device="cuda")
    where = dict(pages=pages, page_size=10, seq=seq, ring=17)

    def step(codes, scales, to):
        fx.idx_write_rows("local", x, codes, scales, at, 1 << 20, gamma=gamma, eps=1e-6, freq=freq, mscale=m, **where)
        fx.idx_read_rows("local", codes, scales, at, 1 << 20, out=to, freq=freq, inverse=True, mscale=1 / m, **where)

    x.normal_(generator=g)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        step(*caches[0], out)
    for c, s in caches:
        c.zero_(), s.zero_()
    want = torch.empty_like(out)
    for i in range(4):
        x.normal_(generator=g)
        at.copy_(torch.tensor([5, 6, 7, 6, 7, 8], device="cuda") + 1000 * i)
        graph.replay()
        step(*caches[1], want)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert torch.equal(caches[0][0], caches[1][0]) and torch.equal(caches[0][1], caches[1][1])
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.default_stream())
        out.fill_(0)
        step(*caches[0], out)
    side.synchronize()
    assert torch.equal(out, want)
