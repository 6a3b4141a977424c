"""Workloads of the caches' operators: rows normalised, rotated, quantised and written to their places in a cache,
rows read back, and attention over the FP8 cache of local positions, joined with the attention over a selection.

`listed()` and `draw()` give the cases, `prepare()` the data a caller has in hand, `run()` one pass
through an operator: in plain torch operations where `own` is false, through the library where it
is true. `exact()` computes the same results in 64 bits from the definitions.
"""
import math

import torch

own = False

NINF = float("-inf")
# values of a row, of a scale's group, code bytes of a row
FORMATS = {"main": (512, 16, 256), "local": (512, 32, 512), "key": (128, 32, 64)}
LOCAL_EXP = (-15, 7)  # a local row's scales: every value is a 16-bit float


def listed():
    return [
        # a decode step of one user: the newest token's row for the cache of local positions, a ring of 256 entries
        dict(name="write one local", op="write", format="local", tokens=1, seqs=1, n=256, dtype="bf16", norm=True, rot=64,
             offset=448, layout="interleaved", page=0, ring=True, pad=0, factor=1.0),
        # a decode step of a batch: one row of each sequence for the paged FP4 cache, in a stretched context
        dict(name="write batch main", op="write", format="main", tokens=64, seqs=64, n=32768, dtype="bf16", norm=True,
             rot=64, offset=448, layout="interleaved", page=64, ring=False, pad=64, factor=32.0),
        # a long prefill chunk of two sequences, rows in 32 bits from a compressor
        dict(name="write chunk main", op="write", format="main", tokens=32770, seqs=2, n=16385, dtype="f32", norm=False,
             rot=64, offset=448, layout="interleaved", page=64, ring=False, pad=0, factor=1.0),
        # a prefill chunk for the cache of local positions
        dict(name="write chunk local", op="write", format="local", tokens=16384, seqs=1, n=16384, dtype="bf16", norm=True,
             rot=64, offset=448, layout="half", page=100, ring=False, pad=64, factor=1.0),
        # the indexer's keys of a prefill chunk
        dict(name="write chunk keys", op="write", format="key", tokens=65537, seqs=1, n=65537, dtype="bf16", norm=True,
             rot=64, offset=0, layout="half", page=0, ring=False, pad=0, factor=1.0),
        # the selected rows of a batch, turned back to their content
        dict(name="read selected main", op="read", format="main", tokens=32768, seqs=64, n=32768, dtype="bf16", rot=64,
             offset=448, layout="interleaved", page=64, ring=False, factor=32.0),
        # the windows of 33 sequences, in 32 bits, as they are stored
        dict(name="read windows local", op="read", format="local", tokens=33 * 128, seqs=33, n=131072, dtype="f32", rot=0,
             offset=0, layout="half", page=0, ring=True, factor=1.0),
        # one user's newest token over its window, joined with the selection's part: latency counts
        dict(name="local one", op="local", seqs=1, new=1, n=131072, heads=64, window=128, page=0, ring=True, join=True,
             turn=True, pad=0),
        # a serving batch, three of its slots idle, windows in pages
        dict(name="local batch", op="local", seqs=64, new=1, n=32768, heads=64, window=128, page=64, ring=True, join=True,
             turn=True, pad=3),
        # a prefill chunk: every query with its own window, joined and turned back
        dict(name="local chunk", op="local", seqs=1, new=4096, n=4224, heads=64, window=128, page=0, ring=False, join=True,
             turn=True, pad=0),
        # draft positions over everything in a long FP8 cache, its length split
        dict(name="local long", op="local", seqs=8, new=3, n=65537, heads=64, window=0, page=64, ring=False, join=False,
             turn=False, pad=0),
        # a chunk over everything visible, pages that end inside a tile
        dict(name="local chunk visible", op="local", seqs=2, new=257, n=16384, heads=64, window=0, page=24, ring=False,
             join=False, turn=True, pad=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("write", "write", "read", "local", "local"))
    page = rng.choice((0, 0, 1, 16, 24, 64, 100, 256))
    if op in ("write", "read"):
        fmt = rng.choice(("main", "local", "key"))
        dim = FORMATS[fmt][0]
        seqs = _log(rng, 1, 64)
        per = _log(rng, 1, 32768 * 512 // dim // seqs)  # tokens of each sequence
        rot = 0 if fmt == "key" and op == "read" else rng.choice((0, 64, 64, 2 * rng.randint(1, dim // 2), dim))
        c = dict(op=op, format=fmt, tokens=seqs * per, seqs=seqs, n=per + _log(rng, 1, 4096) - 1,
                 dtype=rng.choice(("bf16", "f32")), rot=rot, offset=rng.choice((0, dim - rot)),
                 layout=rng.choice(("half", "interleaved")), page=page, ring=rng.random() < 0.3,
                 factor=rng.choice((1.0, 8.0, 40.0)))
        if op == "write":
            c.update(norm=rng.random() < 0.5, pad=rng.choice((0, 64)))
        return c
    heads = rng.choice((1, 5, 8, 16, 32, 64, 64, 100, 128))
    n = _log(rng, 1, 65536)
    if rng.random() < 0.6:
        window = rng.choice((128, 128, _log(rng, 1, 1000)))
        seqs = _log(rng, 1, 128)
        new = min(n, _log(rng, 1, max(1, min((1 << 18) // (seqs * heads), (1 << 20) // (seqs * window)))))
        ring = rng.random() < 0.5
    else:
        window, ring = 0, False
        seqs = _log(rng, 1, min(32, max(1, (1 << 18) // n)))
        new = min(n, _log(rng, 1, max(1, (1 << 28) // (seqs * n * heads))))
    return dict(op=op, seqs=seqs, new=new, n=n, heads=heads, window=window, page=page, ring=ring, join=rng.random() < 0.5,
                turn=rng.random() < 0.5, pad=rng.choice((0, 1)))


# ---------------------------------------------------------------------------- inputs

def _rope_freqs(rot, factor):
    """Rotation per position of each pair; factor > 1 stretches a 4096-token training length by it
    (fast rotations kept, slow ones divided, a linear ramp in rotations between)."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if factor == 1.0:
        return f.cuda(), 1.0
    turns = 4096.0 * f / (2.0 * math.pi)
    keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
    return (f * keep + f / factor * (1.0 - keep)).cuda(), 0.1 * math.log(factor) + 1.0


def _places(st, seqs, entries, ring, g):
    """Where `entries` places of each sequence lie: pages given out at random, or one range after another."""
    page = st["c"]["page"]
    st["ring"] = entries if ring else 0
    st["pages"] = st["starts"] = None
    if page:
        per = -(-entries // page)
        st["pages"] = torch.randperm(seqs * per + 3, device="cuda", generator=g)[:seqs * per].view(seqs, per).int()
        return (seqs * per + 3) * page
    st["starts"] = torch.arange(seqs, device="cuda") * entries
    return seqs * entries


def _stored_rows(fmt, rows, g):
    """A cache of unit-RMS rows in its format: codes and scale bytes."""
    dim, group, width = FORMATS[fmt]
    codes = torch.empty(rows, width, dtype=torch.uint8, device="cuda")
    scales = torch.empty(rows, dim // group, dtype=torch.uint8, device="cuda")
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    for r in range(0, rows, 1 << 18):
        x = torch.randn(min(1 << 18, rows - r), dim // group, group, device="cuda", generator=g)
        top = x.abs().amax(-1)
        if fmt == "local":
            e = torch.ceil(torch.log2(top / 448.0))
            codes[r:r + x.shape[0]] = (x * torch.exp2(-e)[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).flatten(1)
            scales[r:r + x.shape[0]] = (e + 127).to(torch.uint8)
            continue
        if fmt == "main":
            s = (top / 6.0).to(torch.float8_e4m3fn)
            b, s = s.view(torch.uint8), s.float()
        else:
            e = torch.ceil(torch.log2(top / 6.0))
            b, s = (e + 127).to(torch.uint8), torch.exp2(e)
        k = torch.bucketize(x.abs() / s[..., None], mid).to(torch.uint8)
        k |= ((x < 0) & (k > 0)).to(torch.uint8) << 3
        k = k.view(-1, width, 2)
        codes[r:r + x.shape[0]], scales[r:r + x.shape[0]] = k[..., 0] | (k[..., 1] << 4), b
    return codes, scales


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = dict(case)
    st = dict(c=c)
    if c["op"] == "local":
        return _prepare_local(st, g)
    dim, group, width = FORMATS[c["format"]]
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    seqs, tokens = c["seqs"], c["tokens"]
    per = tokens // seqs
    # a ring holds one call's tokens at least, and wraps among them; otherwise a sequence has n entries and the tokens come somewhere
    # in them (a written chunk at the end of what there is, a read list spread over it)
    entries = max(per, 256 if c["ring"] else c["n"])
    rows = _places(st, seqs, entries, c["ring"], g)
    far = torch.randint(0, max(entries - per, c["n"] if c["ring"] else 0) + 1, (seqs, 1), device="cuda", generator=g)
    at = torch.arange(per, device="cuda").expand(seqs, per)
    if c["op"] == "read" and not c["ring"]:
        at = ((at + torch.rand(seqs, per, device="cuda", generator=g, dtype=torch.float64) * 0.999) * entries / per).long()
    else:
        at = at + far
    st["at"] = at.reshape(-1).contiguous()
    st["seq"] = torch.arange(seqs, device="cuda").repeat_interleave(per).int()
    st["base"] = None if st["starts"] is None else st["starts"].repeat_interleave(per)
    st["max_n"] = max(int(c["n"]), entries) + tokens  # entries a sequence may come to have
    if st["pages"] is not None and not c["ring"]:
        st["max_n"] = st["pages"].shape[1] * c["page"]
    st["freq"] = None
    st["mscale"] = 1.0
    if c["rot"]:
        st["freq"], st["mscale"] = _rope_freqs(c["rot"], c["factor"])
    if c["op"] == "read":
        st["codes"], st["scales"] = _stored_rows(c["format"], rows, g)
        st["out"] = torch.empty(tokens, dim, dtype=dt, device="cuda")
        return st
    x = torch.randn(tokens, dim + c["pad"], device="cuda", generator=g)
    x *= torch.exp(0.5 * torch.randn(tokens, 1, device="cuda", generator=g))
    x *= torch.exp(0.7 * torch.randn(dim + c["pad"], device="cuda", generator=g))  # some channels are large
    st["x"] = x.to(dt)[:, c["pad"]:]
    st["gamma"] = (1.0 + 0.1 * torch.randn(dim, device="cuda", generator=g)) if c["norm"] else None
    st["eps"] = 1e-6 if c["norm"] else None
    st["signs"] = None
    if c["format"] == "key":
        st["signs"] = (torch.randint(0, 2, (dim,), device="cuda", generator=g) * 2 - 1).to(torch.int8)
        h2 = torch.tensor([[1.0, 1.0], [1.0, -1.0]], dtype=torch.float64, device="cuda")
        h4 = torch.kron(h2, h2)
        st["hadamard"] = torch.kron(torch.kron(torch.kron(h4, h4), h4), h2)
    st["codes"] = torch.zeros(rows, width, dtype=torch.uint8, device="cuda")
    st["scales"] = torch.zeros(rows, dim // group, dtype=torch.uint8, device="cuda")
    st["out"] = torch.empty(tokens, dim, dtype=torch.bfloat16, device="cuda")
    return st


def _prepare_local(st, g):
    c = st["c"]
    seqs, new, n, heads, window = (c[x] for x in ("seqs", "new", "n", "heads", "window"))
    lens = n - torch.randint(0, (n - new) // 4 + 1, (seqs,), device="cuda", generator=g)
    lens[-1] = n
    nq = seqs * new
    n_vis = (lens[:, None] - new + 1 + torch.arange(new, device="cuda")).reshape(-1)
    if c["pad"] and nq > c["pad"]:
        n_vis[:c["pad"]] = 0
    st["n_vis"] = n_vis.int()
    entries = window + new - 1 if c["ring"] else n
    rows = _places(st, seqs, entries, c["ring"], g)
    st["seq"] = torch.arange(seqs, device="cuda").int()  # of each run of `new` queries
    st["base"] = st["starts"]
    st["codes"], st["scales"] = _stored_rows("local", rows, g)
    st["q"] = (2.0 * torch.randn(nq, heads, 512, device="cuda", generator=g)).bfloat16()
    st["scale"] = 512 ** -0.5
    st["other"] = st["other_lse"] = None
    if c["join"]:  # the part over the selection; a query's head without one now and then
        st["other"] = (0.3 * torch.randn(nq, heads, 512, device="cuda", generator=g)).bfloat16()
        st["other_lse"] = 6.0 + torch.randn(nq, heads, device="cuda", generator=g)
        st["other_lse"][torch.rand(nq, heads, device="cuda", generator=g) < 0.01] = NINF
        st["other_lse"][n_vis == 0] = NINF
    st["freq"], st["mscale"], st["pos"] = None, 1.0, None
    if c["turn"]:
        st["freq"], m = _rope_freqs(64, 32.0)
        st["mscale"] = 1.0 / m
        st["pos"] = (lens[:, None] - new + torch.arange(new, device="cuda")).reshape(-1)
    st["out"] = torch.empty_like(st["q"])
    st["lse"] = torch.empty(nq, heads, device="cuda")
    return st


# ---------------------------------------------------------------------------- plain forms

def _rows_at(st, seq, base, at):
    """Cache rows of entries `at` (all there) of sequences."""
    page = st["c"]["page"]
    if st["ring"]:
        at = at % st["ring"]
    if st["pages"] is None:
        return base + at
    return st["pages"].long()[seq.long(), at // page] * page + at % page


def _turn(x, pos, freq, offset, layout, mscale, back):
    """x [..., dim] with its rotated part turned by pos * freq (broadcast over x's leading axes)."""
    rot = 2 * freq.numel()
    a = pos.double()[..., None] * freq
    cos = (a.cos() * mscale).to(x.dtype)
    sin = (a.sin() * (-mscale if back else mscale)).to(x.dtype)
    part = x[..., offset:offset + rot]
    if layout == "half":
        x0, x1 = part.chunk(2, -1)
        y = torch.cat([x0 * cos - x1 * sin, x1 * cos + x0 * sin], -1)
    else:
        x0, x1 = part[..., 0::2], part[..., 1::2]
        y = torch.stack([x0 * cos - x1 * sin, x1 * cos + x0 * sin], -1).flatten(-2)
    return torch.cat([x[..., :offset], y, x[..., offset + rot:]], -1)


def _pow2(e):
    """2 ** e of whole numbers, exact (exp2 on the GPU need not be)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _fp4_codes(v):
    """E2M1 codes [..., 2m] of values (64 bits, at most 6 in magnitude or cut to it), two to a byte."""
    a = v.abs()
    k = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() + (a > 2.5).byte() +
         (a >= 3.5).byte() + (a > 5.0).byte())
    k = k | (((v < 0) & (k > 0)).byte() << 3)
    k = k.view(*v.shape[:-1], -1, 2)
    return k[..., 0] | (k[..., 1] << 4)


def _plain_rows(fmt, codes, scales):
    """Rows of a cache as float32."""
    dim, group, _ = FORMATS[fmt]
    if fmt == "local":
        x = codes.view(torch.float8_e4m3fn).float()
    else:
        v = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device="cuda")
        v = torch.cat([v, -v])
        x = torch.stack([v[(codes & 15).int()], v[(codes >> 4).int()]], -1).flatten(-2)
    s = scales.view(torch.float8_e4m3fn).float() if fmt == "main" else _pow2(scales.int() - 127).float()
    return (x.view(*x.shape[:-1], dim // group, group) * s[..., None]).flatten(-2)


def _plain_write(st):
    """The rows in 64 bits (a code turns on which side of a border a value lies), quantised, stored and read back."""
    c = st["c"]
    dim, group, _ = FORMATS[c["format"]]
    y = st["x"].double()
    if c["norm"]:
        y = y * (y.square().mean(-1, keepdim=True) + st["eps"]).rsqrt() * st["gamma"].double()
    if c["rot"]:
        y = _turn(y, st["at"], st["freq"], c["offset"], c["layout"], st["mscale"], False)
    if c["format"] == "key":
        y = ((y * st["signs"]) @ st["hadamard"]).float() * torch.tensor(2.0 ** -3.5, device="cuda")
        y = y.double()
    y = y.view(-1, dim // group, group)
    top = y.abs().amax(-1)
    if c["format"] == "main":
        v = top / 6.0
        step = _pow2((torch.frexp(v)[1] - 1).clamp(min=-6) - 3)
        s = (torch.ceil(v / step) * step).clamp(max=448.0)
        stored = s.to(torch.float8_e4m3fn).view(torch.uint8)
        codes = _fp4_codes((y / torch.where(s > 0, s, 1.0)[..., None]).flatten(1))
    else:
        most = 448.0 if c["format"] == "local" else 6.0
        lo, hi = LOCAL_EXP if c["format"] == "local" else (-127, 127)
        m, e = torch.frexp(top / most)  # m in [0.5, 1), or 0
        e = torch.where(top == 0, lo, (e - (m == 0.5).int()).clamp(lo, hi))
        stored = (e + 127).to(torch.uint8)
        v = y * _pow2(-e)[..., None]
        if c["format"] == "local":
            v = v.clamp(-448.0, 448.0)
            step = _pow2((torch.frexp(v)[1] - 1).clamp(min=-6) - 3)
            v = torch.round(v / step) * step + 0.0
            codes = v.float().to(torch.float8_e4m3fn).view(torch.uint8).flatten(1)
        else:
            codes = _fp4_codes(v.flatten(1))
    rows = _rows_at(st, st["seq"], st["base"], st["at"])
    st["codes"][rows] = codes
    st["scales"][rows] = stored
    return _plain_rows(c["format"], st["codes"][rows], st["scales"][rows]).bfloat16()


def _plain_read(st):
    c = st["c"]
    rows = _rows_at(st, st["seq"], st["base"], st["at"])
    x = _plain_rows(c["format"], st["codes"][rows], st["scales"][rows])
    if c["rot"]:
        x = _turn(x, st["at"], st["freq"], c["offset"], c["layout"], 1.0 / st["mscale"], True)
    return x.to(st["out"].dtype)


def _plain_local(st):
    c = st["c"]
    seqs, new, n, heads, window = (c[x] for x in ("seqs", "new", "n", "heads", "window"))
    nv = st["n_vis"].long().view(seqs, new, 1)
    q = st["q"].float() * st["scale"]
    who = torch.arange(seqs, device="cuda").view(seqs, 1, 1)
    start = None if st["base"] is None else st["base"].view(seqs, 1, 1)
    if window:  # each query's own rows
        pos = nv - window + torch.arange(window, device="cuda")
        ok = pos >= 0
        rows = _rows_at(st, who, start, pos.clamp(min=0)).view(seqs * new, window)
        ok, q = ok.view(seqs * new, 1, 1, -1) & (nv.view(-1, 1, 1, 1) > 0), q.view(seqs * new, heads, 512)
    else:
        pos = torch.arange(n, device="cuda").view(1, 1, n)
        ok = (pos < nv).view(seqs, new, 1, n)
        rows = _rows_at(st, who, start, pos)[:, 0]
        q = q.view(seqs, new * heads, 512)
    kv = _plain_rows("local", st["codes"][rows], st["scales"][rows])
    s = torch.bmm(q, kv.transpose(1, 2).contiguous()).view(ok.shape[0], ok.shape[1], heads, -1)
    s = s.masked_fill_(~ok, NINF)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(m.masked_fill(m == NINF, 0.0)).exp_()
    z = p.sum(-1, keepdim=True)
    lse = (m + z.log()).view(st["lse"].shape)
    o = torch.bmm(p.view(p.shape[0], -1, p.shape[-1]), kv).view(*p.shape[:-1], 512)
    o = (o / z.clamp(min=1e-30)).view(st["q"].shape)
    if c["join"]:
        l2 = st["other_lse"]
        top = torch.maximum(lse, l2)
        top = top.masked_fill(top == NINF, 0.0)
        a, b = (lse - top).exp(), (l2 - top).exp()
        o = (o * a[..., None] + st["other"].float() * b[..., None]) / (a + b).clamp(min=1e-30)[..., None]
        lse = top + (a + b).log()
    if c["turn"]:
        o = _turn(o, st["pos"][:, None], st["freq"], 448, "interleaved", st["mscale"], True)
    return {"out": o.bfloat16(), "lse": lse}


def run(st):
    c = st["c"]
    if own:
        import top_fp4_lightning_amd as fx

        if c["op"] == "local":
            if "ws" not in st:
                st["ws"] = fx.workspace(fx.IDX_OP_ATTEND_LOCAL, c["seqs"] * c["new"],
                                        c["window"] + c["new"] - 1 if c["window"] else c["n"], c["heads"])
            fx.idx_attend_local(st["q"], st["codes"], st["scales"], st["n_vis"], c["n"], st["scale"], st["out"], st["ws"],
                                lse=st["lse"], window=c["window"], ring=st["ring"], group=c["new"], kv_base=st["base"],
                                pages=st["pages"], page_size=c["page"], seq=st["seq"], other=st["other"],
                                other_lse=st["other_lse"], pos=st["pos"], freq=st["freq"], layout="interleaved",
                                mscale=st["mscale"])
            return {"out": st["out"], "lse": st["lse"]}
        where = dict(kv_base=st["base"], pages=st["pages"], page_size=c["page"], seq=st["seq"], ring=st["ring"])
        turn = dict(pos=st["at"], freq=st["freq"], offset=c["offset"], layout=c["layout"])
        if c["op"] == "read":
            return fx.idx_read_rows(c["format"], st["codes"], st["scales"], st["at"], st["max_n"], out=st["out"], inverse=True,
                                    mscale=1.0 / st["mscale"], **where, **turn)
        fx.idx_write_rows(c["format"], st["x"], st["codes"], st["scales"], st["at"], st["max_n"], gamma=st["gamma"],
                          eps=st["eps"], signs=st["signs"], mscale=st["mscale"], **where, **turn)
        return fx.idx_read_rows(c["format"], st["codes"], st["scales"], st["at"], st["max_n"], out=st["out"], **where)
    return {"write": _plain_write, "read": _plain_read, "local": _plain_local}[c["op"]](st)


def work(case):
    c = case
    if c["op"] == "local":
        nq, window, new = c["seqs"] * c["new"], c["window"], c["new"]
        length = c["n"] - (c["n"] - new) / 8 - (new - 1) / 2  # mean visible positions
        entries = min(length, window or length)
        rows = c["seqs"] * min(c["n"], entries + new - 1)
        pairs = nq * c["heads"]
        return {"bytes": 528 * rows + pairs * 512 * 2 * (3 if c["join"] else 2) + pairs * 4 * (2 if c["join"] else 1)
                + 12 * nq, "flops": 4 * pairs * entries * 512}
    dim, group, width = FORMATS[c["format"]]
    row, size = width + dim // group, 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "read":
        return {"bytes": c["tokens"] * (row + size * dim + 12), "flops": c["tokens"] * (dim + 3 * c["rot"])}
    # the rows in, the stored rows out; read back, 16-bit values out
    mix = 7 * dim if c["format"] == "key" else 0
    return {"bytes": c["tokens"] * (size * dim + 2 * row + 2 * dim + 12),
            "flops": c["tokens"] * ((4 if c["norm"] else 0) * dim + 3 * c["rot"] + mix + 3 * dim)}


# ---------------------------------------------------------------------------- 64 bits, from the definitions

def _nearest(v, table):
    """Nearest entry of an ascending table of values >= 0 to each |v|, a tie to the even place; keeps the sign."""
    mid = (table[1:] + table[:-1]) / 2
    i = torch.searchsorted(mid, v.abs().contiguous())  # middles below |v|
    tie = (i < len(mid)) & (mid[i.clamp(max=len(mid) - 1)] == v.abs()) & (i % 2 == 1)
    return table[i + tie.long()] * torch.sign(v)


def _table(values):
    return torch.tensor(values, device="cuda", dtype=torch.float64)


def _e4m3_table():
    return _table([b * 2.0 ** -9 if b < 8 else (1 + b % 8 / 8) * 2.0 ** (b // 8 - 7) for b in range(127)])


def _e2m1_table():
    return _table([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _exact_rows(fmt, codes, scales):
    dim, group, _ = FORMATS[fmt]
    if fmt == "local":
        t = _e4m3_table()
        t = torch.cat([t, t[:1] * math.nan])
        v = torch.cat([t, -t])[codes.long()]
    else:
        nib = torch.stack([codes % 16, codes // 16], -1).flatten(-2).long()
        v = torch.cat([_e2m1_table(), -_e2m1_table()])[nib]
    if fmt == "main":
        t = _e4m3_table()
        s = torch.cat([t, t[:1] * math.nan, -t, t[:1] * math.nan])[scales.long()]
    else:
        s = _table([2.0 ** (b - 127) for b in range(256)])[scales.long()]
    return v * s.repeat_interleave(group, -1)


def _exact_turn(x, a, offset, layout, m):
    rot = 2 * a.shape[-1]
    x = x.clone()
    part = x[..., offset:offset + rot]
    z = torch.complex(*(p.contiguous() for p in part.chunk(2, -1))) if layout == "half" else torch.view_as_complex(
        part.reshape(*part.shape[:-1], -1, 2))
    z = z * torch.polar(torch.full_like(a, m), a)
    x[..., offset:offset + rot] = torch.cat([z.real, z.imag], -1) if layout == "half" else torch.view_as_real(z).flatten(-2)
    return x


def _exact_places(st):
    """Row of every entry `at`, by its definition."""
    e = st["at"] % st["ring"] if st["ring"] else st["at"]
    if st["pages"] is None:
        return st["starts"][st["seq"].long()] + e
    page = st["c"]["page"]
    table = st["pages"].long()
    return table.flatten()[st["seq"].long() * table.shape[1] + e // page] * page + e % page


def _exact_write(st):
    c = st["c"]
    dim, group, _ = FORMATS[c["format"]]
    y = st["x"].to(torch.float64)
    if c["norm"]:
        y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / dim + st["eps"]) * st["gamma"]
    if c["rot"]:
        y = _exact_turn(y, st["at"].double()[:, None] * st["freq"], c["offset"], c["layout"], st["mscale"])
    if c["format"] == "key":
        i = torch.arange(128, device="cuda")
        odd = torch.zeros(128, 128, dtype=torch.long, device="cuda")
        for b in range(7):
            odd += ((i[:, None] & i[None, :]) >> b) & 1
        y = (st["signs"].double() * y) @ (1.0 - 2.0 * (odd % 2)).double()
        y = (y.float() * torch.tensor(2.0 ** -3.5, device="cuda")).double()  # the definition's two roundings
    y = y.view(-1, dim // group, group)
    top = y.abs().amax(-1)
    if c["format"] == "main":
        t = _e4m3_table()
        s = t[torch.searchsorted(6.0 * t, top.contiguous()).clamp(max=126)]
        v = _nearest(y / torch.where(s > 0, s, 1.0)[..., None], _e2m1_table())
    else:
        most, (lo, hi) = (448.0, LOCAL_EXP) if c["format"] == "local" else (6.0, (-127, 127))
        t = _table([2.0 ** e for e in range(lo, hi + 1)])
        s = t[torch.searchsorted(most * t, top.contiguous()).clamp(max=hi - lo)]
        v = _nearest(y / s[..., None], _e4m3_table() if c["format"] == "local" else _e2m1_table())
    return (v * s[..., None]).flatten(1)


def _exact_local(st):
    c = st["c"]
    new, heads, window = c["new"], c["heads"], c["window"]
    nv = st["n_vis"].tolist()
    first = None if st["starts"] is None else st["starts"].tolist()
    outs = torch.zeros(len(nv), heads, 512, dtype=torch.float64, device="cuda")
    lses = torch.full((len(nv), heads), NINF, dtype=torch.float64, device="cuda")
    for b in range(c["seqs"]):
        seen = nv[b * new:(b + 1) * new]
        low = min((max(0, x - window) if window else 0) for x in seen)
        e = torch.arange(low, max(seen), device="cuda")
        place = e % st["ring"] if st["ring"] else e
        rows = place + first[b] if first is not None else st["pages"][b].long()[place // c["page"]] * c["page"] + place % c["page"]
        kv = _exact_rows("local", st["codes"][rows], st["scales"][rows])
        for t in range(b * new, (b + 1) * new):
            if nv[t] <= 0:
                continue
            mine = kv[(max(0, nv[t] - window) if window else 0) - low:nv[t] - low]
            s = st["scale"] * (st["q"][t].double() @ mine.T)
            lses[t] = torch.logsumexp(s, -1)
            outs[t] = (s - lses[t][:, None]).exp() @ mine
    if c["join"]:
        both = torch.logaddexp(lses, st["other_lse"].double())
        w1 = torch.where(lses == NINF, 0.0, (lses - both).exp())
        w2 = torch.where(st["other_lse"] == NINF, 0.0, (st["other_lse"].double() - both).exp())
        outs, lses = w1[..., None] * outs + w2[..., None] * st["other"].double(), both
    if c["turn"]:
        a = -(st["pos"].double()[:, None] * st["freq"])
        outs = _exact_turn(outs, a[:, None, :].expand(-1, heads, -1), 448, "interleaved", st["mscale"])
    return {"out": outs, "lse": lses}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "local":
        return _exact_local(st)
    if case["op"] == "write":
        return _exact_write(st)
    c = case
    rows = _exact_places(st)
    x = _exact_rows(c["format"], st["codes"][rows], st["scales"][rows])
    if c["rot"]:
        x = _exact_turn(x, -(st["at"].double()[:, None] * st["freq"]), c["offset"], c["layout"], 1.0 / st["mscale"])
    return x
