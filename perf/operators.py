"""Workloads of the attention-side operators: rotary positions, attention over the FP4 main-KV
cache, its weights per position, and the distillation of the indexer's scores.

`listed()` and `draw()` give the cases, `prepare()` the data a caller has in hand, `run()` one pass
through an operator: in plain torch operations where `own` is false, through the library where it
is true. `exact()` computes the same results in 64 bits from the definitions.
"""
import math

import torch

own = False

D = 512  # values of a main-KV row
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
NINF = float("-inf")


def listed():
    return [
        # a decode step's indexer query, 32 heads of 128, one token deep in a scaled context
        dict(name="rope one token", op="rope", tokens=1, heads=32, dim=128, rot=64, offset=0, layout="half",
             dtype="bf16", inverse=False, far=1048576, factor=32.0),
        # the core queries of a prefill chunk: 64 heads of 512, the last 64 values carry the position
        dict(name="rope chunk", op="rope", tokens=4096, heads=64, dim=512, rot=64, offset=448, layout="interleaved",
             dtype="bf16", inverse=False, far=131072, factor=1.0),
        # single-user decode over the layer's selection: latency counts
        dict(name="attend one selected", op="attend", seqs=1, new=1, n=131072, heads=64, k=512, window=0, page=0, pad=0),
        # a serving batch, three of its slots idle, over a paged cache
        dict(name="attend batch selected", op="attend", seqs=64, new=1, n=32768, heads=64, k=512, window=0, page=64,
             pad=3),
        # a prefill chunk, every query with its own selection
        dict(name="attend chunk selected", op="attend", seqs=1, new=4096, n=131072, heads=64, k=512, window=0, page=0,
             pad=0),
        # chunked prefill of layers that attend to everything visible; pages that end inside a tile
        dict(name="attend chunk visible", op="attend", seqs=2, new=257, n=16384, heads=64, k=0, window=0, page=24,
             pad=0),
        # long-context decode over everything visible
        dict(name="attend long visible", op="attend", seqs=8, new=1, n=131072, heads=64, k=0, window=0, page=64, pad=0),
        # the teacher of a small batch: weights at the selected positions
        dict(name="weights batch selected", op="weights", seqs=64, new=1, n=32768, heads=64, k=512, page=64),
        # dense warm-up: the weight of every visible position
        dict(name="weights chunk visible", op="weights", seqs=1, new=1021, n=4096, heads=64, k=0, page=0),
        # the loss of a few short rows
        dict(name="distill few", op="distill", rows=5, n=1001, k=64, masked=0.0, temp=1.0),
        # a training chunk: one row per query
        dict(name="distill chunk", op="distill", rows=4096, n=32768, k=512, masked=0.25, temp=2.0),
        # few queries over the longest rows
        dict(name="distill long", op="distill", rows=8, n=1048576, k=512, masked=0.0, temp=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope", "attend", "attend", "weights", "distill"))
    if op == "rope":
        dim = rng.choice((64, 96, 128, 130, 512))
        rot = rng.choice((dim, 2 * rng.randint(1, dim // 2), dim // 2 // 2 * 2))
        heads = rng.choice((1, 3, 16, 32, 64))
        return dict(op="rope", tokens=_log(rng, 1, 4096 * 64 * 512 // (heads * dim) // 2), heads=heads, dim=dim, rot=rot,
                    offset=rng.choice((0, dim - rot)), layout=rng.choice(("half", "interleaved")),
                    dtype=rng.choice(("bf16", "f32")), inverse=rng.random() < 0.5, far=_log(rng, 1, 1 << 24),
                    factor=rng.choice((1.0, 8.0, 40.0)))
    if op == "distill":
        n = _log(rng, 1, 262144)
        rows = _log(rng, 1, max(1, min(4096, (1 << 26) // n)))
        return dict(op="distill", rows=rows, n=n, k=_log(rng, 1, min(2048, n)), masked=rng.choice((0.0, 0.25, 0.9)),
                    temp=rng.choice((0.5, 1.0, 3.0)))
    heads = rng.choice((1, 5, 8, 16, 32, 64, 64, 100, 128))
    page = rng.choice((0, 1, 16, 24, 64, 100, 256))
    n = _log(rng, 1, 65536)
    if rng.random() < 0.6:  # selected positions
        k = _log(rng, 1, 2048)
        seqs = _log(rng, 1, min(64, max(1, (1 << 20) // n)))
        new = min(n, _log(rng, 1, max(1, (1 << 19) // (seqs * k))))
    else:
        k = 0
        seqs = _log(rng, 1, min(32, max(1, (1 << 18) // n)))
        new = min(n, _log(rng, 1, max(1, (1 << 21) // (seqs * n))))
    c = dict(op=op, seqs=seqs, new=new, n=n, heads=heads, k=k, page=page)
    if op == "attend":
        c.update(window=rng.choice((0, 0, 128, 1000)) if k == 0 else 0, pad=rng.choice((0, 1)))
    return c


# ---------------------------------------------------------------------------- inputs

def _quantised_rows(rows, g):
    """Unit-RMS rows in the main-KV format: codes [rows, 256], E4M3 scale bytes [rows, 32]."""
    codes = torch.empty(rows, D // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(rows, D // 16, dtype=torch.uint8, device="cuda")
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    for r in range(0, rows, 1 << 18):
        x = torch.randn(min(1 << 18, rows - r), D // 16, 16, device="cuda", generator=g)
        s = (x.abs().amax(-1) / 6.0).to(torch.float8_e4m3fn)
        c = torch.bucketize(x.abs() / s.float().clamp(min=2.0 ** -9)[..., None], mid).to(torch.uint8)
        c |= ((x < 0) & (c > 0)).to(torch.uint8) << 3
        c = c.view(-1, D // 2, 2)
        codes[r:r + c.shape[0]] = c[..., 0] | (c[..., 1] << 4)
        scales[r:r + c.shape[0]] = s.view(torch.uint8)
    return codes, scales


def _rope_freqs(rot, factor):
    """Rotation per position of each pair; factor > 1 stretches a 4096-token training length by it
    (fast rotations kept, slow ones divided, a linear ramp in rotations between)."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if factor == 1.0:
        return f.cuda(), 1.0
    turns = 4096.0 * f / (2.0 * math.pi)
    keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
    return (f * keep + f / factor * (1.0 - keep)).cuda(), 0.1 * math.log(factor) + 1.0


def _spread(rows, k, n_vis, g):
    """k distinct ascending positions over each row's visible range (0 .. k-1 where it is shorter)."""
    u = torch.rand(rows, k, device="cuda", generator=g, dtype=torch.float64) * 0.999
    i = ((torch.arange(k, device="cuda") + u) * n_vis[:, None] / k).long()
    return torch.where(n_vis[:, None] >= k, i, torch.arange(k, device="cuda"))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = dict(case)
    if c["op"] == "rope":
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        x = torch.randn(c["tokens"], c["heads"], c["dim"], device="cuda", generator=g).to(dt)
        first = torch.randint(0, c["far"] + 1, (1,), device="cuda", generator=g)
        freq, mscale = _rope_freqs(c["rot"], c["factor"])
        return dict(c=c, x=x, pos=first + torch.arange(c["tokens"], device="cuda"), freq=freq, mscale=mscale,
                    out=torch.empty_like(x))
    if c["op"] == "distill":
        rows, n, k = c["rows"], c["n"], c["k"]
        s = 3.0 * torch.randn(rows, n, device="cuda", generator=g)
        if c["masked"]:  # a pool of 8-position blocks: -inf outside, the newest block always inside
            nb = (n + 7) // 8
            off = torch.rand(rows, nb, device="cuda", generator=g) < c["masked"]
            off[:, -1] = False
            s.masked_fill_(off.repeat_interleave(8, 1)[:, :n], NINF)
        n_vis = n - torch.randint(0, n // 4 + 1, (rows,), device="cuda", generator=g)
        n_vis[0] = n
        if rows > 4:
            n_vis[3] = 0  # a padded row
        i = _spread(rows, k, n_vis, g)
        t = 2.0 * torch.randn(rows, k, device="cuda", generator=g)
        return dict(c=c, scores=s, n_vis=n_vis.int(), t_idx=torch.where(i < n_vis[:, None], i, -1).int(), t_logit=t,
                    dloss=torch.rand(rows, device="cuda", generator=g) / rows, dscores=torch.zeros_like(s),
                    loss=torch.empty(rows, device="cuda"), lse=torch.empty(rows, device="cuda"),
                    t_lse=torch.empty(rows, device="cuda"))
    seqs, new, n, heads, k, page = (c[x] for x in ("seqs", "new", "n", "heads", "k", "page"))
    lens = n - torch.randint(0, (n - new) // 4 + 1, (seqs,), device="cuda", generator=g)
    lens[-1] = n
    nq = seqs * new
    n_vis = (lens[:, None] - new + 1 + torch.arange(new, device="cuda")).reshape(-1)
    if c.get("pad", 0) and nq > c["pad"]:
        n_vis[:c["pad"]] = 0
    st = dict(c=c, n_vis=n_vis.int(), scale=D ** -0.5, kv_base=None, pages=None, seq=None)
    if page:
        per = -(-n // page)
        st["pages"] = torch.randperm(seqs * per + 3, device="cuda", generator=g)[:seqs * per].view(seqs, per).int()
        st["seq"] = torch.arange(seqs, device="cuda").repeat_interleave(new).int()
        rows = (seqs * per + 3) * page
    else:
        st["kv_base"] = (torch.arange(seqs, device="cuda") * n).repeat_interleave(new)
        rows = seqs * n
    st["codes"], st["scales"] = _quantised_rows(rows, g)
    st["q"] = (2.0 * torch.randn(nq, heads, D, device="cuda", generator=g)).bfloat16()
    st["idx"] = None
    if k:
        i = _spread(nq, k, n_vis, g)
        st["idx"] = torch.where(i < n_vis[:, None], i, -1).int()
    st["lse"] = torch.empty(nq, heads, device="cuda")
    if c["op"] == "attend":
        st["out"] = torch.empty_like(st["q"])
    else:
        st["lse"] = _plain_attend(st, want="lse")
        st["weights"] = torch.zeros(nq, k or n, device="cuda")
    return st


# ---------------------------------------------------------------------------- plain forms

def _rows_of(st, pos):
    """Cache rows of positions [seqs, new, m] (all valid)."""
    c = st["c"]
    if st["pages"] is None:
        return st["kv_base"].view(c["seqs"], c["new"], 1) + pos
    p = st["pages"].long()[:, None, :].expand(-1, pos.shape[1], -1)
    return torch.gather(p, 2, pos // c["page"]) * c["page"] + pos % c["page"]


def _plain_kv(st, rows):
    """Main-KV rows as float32 [..., 512]."""
    v = torch.tensor(E2M1 + tuple(-x for x in E2M1), device="cuda")
    pair = torch.stack([v.repeat(16), v.repeat_interleave(16)], 1)  # the two values of a byte
    r = rows.reshape(-1)
    x = pair[st["codes"][r].int()].view(-1, D // 16, 16)
    x = x * st["scales"][r].view(torch.float8_e4m3fn).float()[..., None]
    return x.view(*rows.shape, D)


def _plain_logits(st):
    """(kv, logits, valid) batched over queries (selected) or sequences (visible): kv [b, m, 512],
    logits [b, q, heads, m]."""
    c = st["c"]
    seqs, new, n, heads = c["seqs"], c["new"], c["n"], c["heads"]
    nv = st["n_vis"].long().view(seqs, new, 1)
    q = st["q"].float() * st["scale"]
    if st["idx"] is not None:
        pos = st["idx"].long().view(seqs, new, -1)
        ok = (pos >= 0) & (pos < nv)
        kv = _plain_kv(st, _rows_of(st, pos.clamp(min=0)).view(seqs * new, -1))
        ok, q = ok.view(seqs * new, 1, 1, -1), q.view(seqs * new, heads, D)
    else:
        pos = torch.arange(n, device="cuda").view(1, 1, n)
        ok = pos < nv
        if c.get("window"):
            ok = ok & (pos >= nv - c["window"])
        kv = _plain_kv(st, _rows_of(st, pos.expand(seqs, 1, n) if st["pages"] is not None else
                                    pos.expand(seqs, new, n))[:, 0])
        ok, q = ok.view(seqs, new, 1, n), q.view(seqs, new * heads, D)
    s = torch.bmm(q, kv.transpose(1, 2)).view(ok.shape[0], ok.shape[1], heads, -1)
    return kv, s.masked_fill(~ok, NINF), ok


def _plain_attend(st, want=""):
    kv, s, _ = _plain_logits(st)
    m = s.amax(-1, keepdim=True)
    p = (s - m.masked_fill(m == NINF, 0.0)).exp_()
    z = p.sum(-1, keepdim=True)
    lse = (m + z.log()).view(st["lse"].shape)
    if want == "lse":
        return lse
    o = torch.bmm(p.view(p.shape[0], -1, p.shape[-1]), kv).view(*p.shape[:-1], D)
    return {"out": (o / z.clamp(min=1e-30)).view(st["q"].shape).bfloat16(), "lse": lse}


def _plain_weights(st):
    _, s, ok = _plain_logits(st)
    lse = st["lse"].view(*s.shape[:-1], 1)
    w = (s - lse.masked_fill(lse == NINF, 0.0)).exp_().masked_fill_(~ok, 0.0).mean(2)
    return w.view(st["weights"].shape)


def _plain_rope(st):
    c, x = st["c"], st["x"]
    a = st["pos"].double()[:, None] * st["freq"]
    cos = (a.cos() * st["mscale"]).float()[:, None, :]
    sin = (a.sin() * (-st["mscale"] if c["inverse"] else st["mscale"])).float()[:, None, :]
    part = x[..., c["offset"]:c["offset"] + c["rot"]].float()
    if c["layout"] == "half":
        x0, x1 = part.chunk(2, -1)
        y = torch.cat([x0 * cos - x1 * sin, x1 * cos + x0 * sin], -1)
    else:
        x0, x1 = part[..., 0::2], part[..., 1::2]
        y = torch.stack([x0 * cos - x1 * sin, x1 * cos + x0 * sin], -1).flatten(-2)
    return torch.cat([x[..., :c["offset"]], y.to(x.dtype), x[..., c["offset"] + c["rot"]:]], -1)


def _plain_distill(st):
    c, inv = st["c"], 1.0 / st["c"]["temp"]
    nv = st["n_vis"].long()[:, None]
    seen = torch.arange(c["n"], device="cuda") < nv
    s = (st["scores"] * inv).masked_fill(~seen, NINF)
    m = s.amax(-1, keepdim=True).clamp(min=-3e38)
    lse = m + (s - m).exp().sum(-1, keepdim=True).log()
    i = st["t_idx"].long()
    at = s.gather(1, i.clamp(min=0))
    t = (st["t_logit"] * inv).masked_fill((i < 0) | (i >= nv) | (at == NINF), NINF)
    tm = t.amax(-1, keepdim=True).clamp(min=-3e38)
    e = (t - tm).exp()
    z = e.sum(-1, keepdim=True)
    p = e / z.clamp(min=1e-30)
    live = z > 0
    term = p * ((t - tm - z.log()) - (at - lse))
    loss = term.masked_fill(p == 0, 0.0).sum(-1)
    d = (s - lse).exp().scatter_add_(1, i.clamp(min=0), -p)
    d = (d * (st["dloss"][:, None] * inv)).masked_fill(~(live & (s > NINF)), 0.0)
    return {"loss": loss, "dscores": d}


def run(st):
    c = st["c"]
    if own:
        import top_fp4_lightning_amd as fx

        if c["op"] == "rope":
            return fx.idx_rope(st["x"], st["pos"], st["freq"], offset=c["offset"], layout=c["layout"],
                               mscale=st["mscale"], inverse=c["inverse"], out=st["out"])
        if c["op"] == "distill":
            if "ws" not in st:
                st["ws"] = fx.workspace(fx.IDX_OP_DISTILL, c["rows"], c["n"], 1)
            fx.idx_distill(st["scores"], st["n_vis"], c["n"], st["t_idx"], st["t_logit"], st["loss"], st["lse"],
                           st["t_lse"], st["ws"], inv_temp=1.0 / c["temp"])
            fx.idx_distill_bwd(st["scores"], st["n_vis"], c["n"], st["t_idx"], st["t_logit"], st["lse"], st["t_lse"],
                               st["dloss"], st["dscores"], inv_temp=1.0 / c["temp"])
            return {"loss": st["loss"], "dscores": st["dscores"]}
        where = dict(kv_base=st["kv_base"], pages=st["pages"], page_size=c["page"], seq=st["seq"], idx=st["idx"])
        if c["op"] == "weights":
            return fx.idx_attend_weights(st["q"], st["codes"], st["scales"], st["n_vis"], c["n"], st["scale"], st["lse"],
                                         st["weights"], **where)
        if "ws" not in st:
            st["ws"] = fx.workspace(fx.IDX_OP_ATTEND, st["q"].shape[0], c["k"] or c["n"], c["heads"])
        fx.idx_attend(st["q"], st["codes"], st["scales"], st["n_vis"], c["n"], st["scale"], st["out"], st["ws"],
                      lse=st["lse"], window=c["window"], **where)
        return {"out": st["out"], "lse": st["lse"]}
    return {"rope": _plain_rope, "attend": _plain_attend, "weights": _plain_weights, "distill": _plain_distill}[c["op"]](st)


def work(case):
    c = case
    if c["op"] == "rope":
        size = 2 if c["dtype"] == "bf16" else 4
        return {"bytes": 2 * size * c["tokens"] * c["heads"] * c["dim"] + 8 * c["tokens"] + 4 * c["rot"],
                "flops": 3 * c["tokens"] * c["heads"] * c["rot"]}
    if c["op"] == "distill":
        # lengths are spread evenly over the last quarter of the row; the row is read for the loss, read and
        # written for the gradient
        return {"bytes": 12 * 0.875 * c["rows"] * c["n"] + 16 * c["rows"] * c["k"], "flops": 8 * 0.875 * c["rows"] * c["n"]}
    nq = c["seqs"] * c["new"]
    length = c["n"] - (c["n"] - c["new"]) / 8 - (c["new"] - 1) / 2  # mean visible positions
    if c["k"]:
        entries = min(c["k"], length)
        rows = min(nq * entries, c["seqs"] * c["n"])
    else:
        entries = min(length, c.get("window") or length)
        rows = c["seqs"] * min(c["n"], entries + c["new"] - 1)
    io = 2 if c["op"] == "attend" else 1
    return {"bytes": 288 * rows + io * nq * c["heads"] * D * 2 + 4 * nq * c["heads"] + 4 * nq * c["k"]
            + (4 * nq * entries if io == 1 else 0), "flops": 2 * io * nq * c["heads"] * entries * D}


# ---------------------------------------------------------------------------- 64 bits, from the definitions

def _exact_kv(st, rows):
    b = st["codes"][rows]
    nib = torch.stack([b & 15, b >> 4], -1).flatten(-2).double()
    mag = nib % 8
    e = (mag / 2).floor()  # exponent field; field 0 is the subnormal step of a half
    v = torch.where(e == 0, mag / 2, (1 + (mag % 2) / 2) * 2.0 ** (e - 1)) * torch.where(nib >= 8, -1.0, 1.0)
    s = st["scales"][rows].double()
    f = ((s % 128) / 8).floor()
    s = torch.where(f == 0, (s % 8) * 2.0 ** -9, (1 + (s % 8) / 8) * 2.0 ** (f - 7)) * torch.where(s >= 128, -1.0, 1.0)
    return v * s.repeat_interleave(16, -1)


def _exact_attention(st):
    c = st["c"]
    seqs, new, heads, n = c["seqs"], c["new"], c["heads"], c["n"]
    nv = st["n_vis"].tolist()
    base = None if st["kv_base"] is None else st["kv_base"].tolist()
    outs, lses = [], []
    weights = None if c["op"] == "attend" else torch.zeros(st["weights"].shape, dtype=torch.float64, device="cuda")
    for b in range(seqs):
        whole = None
        for i in range(new):
            t = b * new + i
            if st["idx"] is not None:
                slot = ((st["idx"][t] >= 0) & (st["idx"][t] < nv[t])).nonzero()[:, 0]
                pos = st["idx"][t][slot].long()
            else:
                slot = pos = torch.arange(max(0, nv[t] - c["window"]) if c.get("window") else 0, nv[t], device="cuda")
            if st["idx"] is None and new > 1:
                if whole is None:
                    everything = torch.arange(n, device="cuda")
                    whole = _exact_kv(st, everything + base[t] if base else
                                      st["pages"][b].long()[everything // c["page"]] * c["page"] + everything % c["page"])
                kv = whole[int(pos[0]):int(pos[-1]) + 1] if len(pos) else whole[:0]
            else:
                kv = _exact_kv(st, pos + base[t] if base else
                               st["pages"][b].long()[pos // c["page"]] * c["page"] + pos % c["page"])
            s = st["scale"] * (st["q"][t].double() @ kv.T)
            if weights is not None:
                if len(pos):
                    weights[t, slot] = (s - st["lse"][t].double()[:, None]).exp().mean(0)
                continue
            lse = torch.logsumexp(s, -1) if len(pos) else torch.full((heads,), NINF, dtype=torch.float64, device="cuda")
            lses.append(lse)
            outs.append((s - lse[:, None]).exp() @ kv if len(pos) else torch.zeros(heads, D, dtype=torch.float64, device="cuda"))
    return weights if weights is not None else {"out": torch.stack(outs), "lse": torch.stack(lses)}


def exact(case, seed):
    st = prepare(case, seed)
    c = case
    if c["op"] == "rope":
        a = st["pos"].double()[:, None] * st["freq"] * (-1.0 if c["inverse"] else 1.0)
        x = st["x"].double()
        part = x[..., c["offset"]:c["offset"] + c["rot"]]
        z = torch.complex(*part.chunk(2, -1)) if c["layout"] == "half" else torch.view_as_complex(
            part.reshape(*part.shape[:-1], -1, 2))
        z = z * torch.polar(torch.full_like(a, st["mscale"]), a)[:, None, :]
        y = torch.cat([z.real, z.imag], -1) if c["layout"] == "half" else torch.view_as_real(z).flatten(-2)
        x[..., c["offset"]:c["offset"] + c["rot"]] = y
        return x
    if c["op"] != "distill":
        return _exact_attention(st)
    loss = torch.zeros(c["rows"], dtype=torch.float64, device="cuda")
    grad = torch.zeros(c["rows"], c["n"], dtype=torch.float64, device="cuda")
    nv = st["n_vis"].tolist()
    for r in range(c["rows"]):
        s = st["scores"][r, :nv[r]].double() / c["temp"]
        at = st["t_idx"][r].long()
        keep = (at >= 0) & (at < nv[r])
        at, t = at[keep], st["t_logit"][r].double()[keep] / c["temp"]
        there = s[at] > NINF
        at, t = at[there], t[there]
        if not len(at):
            continue
        logp, logq = torch.log_softmax(t, -1), torch.log_softmax(s, -1)
        loss[r] = (logp.exp() * (logp - logq[at])).sum()
        d = logq.exp()
        d.index_add_(0, at, -logp.exp())
        grad[r, :nv[r]] = d * float(st["dloss"][r]) / c["temp"]
    return {"loss": loss, "dscores": grad}
