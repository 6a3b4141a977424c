"""Rotary positions (idx_rope) against the definition in extended precision."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fx():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import top_fp4_lightning_amd

    return top_fp4_lightning_amd


def reference(x, pos, freq, offset, layout, mscale, inverse):
    """(y, size of the terms) in extended precision: x [tokens, heads, dim]"""
    pi2 = 2 * np.longdouble("3.14159265358979323846264338327950288")
    a = np.fmod(np.asarray(pos, np.longdouble)[:, None] * np.asarray(freq, np.longdouble), pi2)
    c, s = np.cos(a)[:, None], np.sin(a)[:, None]
    if inverse:
        s = -s
    half = len(freq)
    at = np.arange(half)
    i0, i1 = (at, at + half) if layout == "half" else (2 * at, 2 * at + 1)
    x = np.asarray(x, np.longdouble)
    y, size = x.copy(), np.zeros_like(x)
    x0, x1 = x[..., offset + i0], x[..., offset + i1]
    y[..., offset + i0] = mscale * (x0 * c - x1 * s)
    y[..., offset + i1] = mscale * (x1 * c + x0 * s)
    size[..., offset + i0] = size[..., offset + i1] = abs(mscale) * (abs(x0) + abs(x1))
    return y.astype(np.float64), size.astype(np.float64)


def tolerance(y, size, dtype):
    """fp32 arithmetic: the remainder of the turns rounds by 2^-25 of a turn (2^-22.3 rad), sin and cos by 2^-23,
    their product with mscale, the two products and the sum by 2^-24 each: below 2^-21 of the terms. Then half a step."""
    return 2.0 ** -21 * size + (2.0 ** -8 * np.abs(y) if dtype == torch.bfloat16 else 0.0)


def run_case(fx, shape, rot, offset, layout, dtype, inverse=False, far=1000, mscale=1.0, in_place=False, x=None, out=None,
             base=10000.0, pos=None):
    rng = np.random.default_rng(sum(shape) + rot)
    tokens, heads, dim = shape
    if x is None:
        x = torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(dtype).cuda()
    freq, one = fx.rope_freqs(rot, base)
    assert one == 1.0
    pos = np.asarray(pos if pos is not None else rng.integers(0, far + 1, tokens), np.int64)
    want, size = reference(x.double().cpu().numpy(), pos, freq.cpu().numpy(), offset, layout, mscale, inverse)
    print(f"rope {shape} rot={rot} offset={offset} {layout} {dtype} in_place={in_place}", flush=True)
    got = fx.idx_rope(x, torch.from_numpy(pos).cuda(), freq, offset=offset, layout=layout, mscale=mscale,
                      inverse=inverse, out=x if in_place else out)
    got = got.double().cpu().numpy()
    assert (np.abs(got - want) <= tolerance(want, size, dtype)).all(), np.abs(got - want).max()
    return got


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("tokens,heads,dim,rot,offset", [
    (1, 1, 2, 2, 0), (1, 32, 128, 64, 0), (3, 32, 128, 64, 64), (5, 64, 512, 64, 448), (700, 1, 512, 64, 448),
    (33, 3, 130, 66, 7), (4, 5, 130, 130, 0), (9, 2, 96, 8, 8), (2, 7, 24, 16, 8), (2000, 2, 16, 16, 0),
    (3, 1, 8192, 8192, 0), (17, 300, 4, 2, 1)])
def test_shapes(fx, tokens, heads, dim, rot, offset, layout, dtype):
    for inverse in (False, True):
        for in_place in (False, True):
            run_case(fx, (tokens, heads, dim), rot, offset, layout, dtype, inverse, in_place=in_place, mscale=1.25)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("heads,dim,rot,offset", [
    (3, 96, 2, 0), (3, 96, 2, 94), (5, 128, 18, 16), (5, 128, 8, 8), (3, 128, 16, 16), (2, 100, 20, 40), (7, 130, 64, 66),
    (1, 512, 512, 0), (2, 516, 256, 0), (2, 520, 64, 456), (1, 1024, 64, 960), (4, 66, 4, 2), (3, 65, 6, 1)])
def test_widths_of_access(fx, heads, dim, rot, offset, layout, dtype):
    """sizes that allow 16, 8 or 4 bytes or one value, halves of odd length, rows of more and of fewer vectors than a
    wavefront has lanes; whole and in place, at an odd address, too"""
    for in_place in (False, True):
        run_case(fx, (23, heads, dim), rot, offset, layout, dtype, in_place=in_place, mscale=0.75)
    room = torch.randn(23 * heads * dim + 1, device="cuda").to(dtype)
    x = room[1:].view(23, heads, dim)
    run_case(fx, (23, heads, dim), rot, offset, layout, dtype, x=x, inverse=True)


@pytest.mark.parametrize("far", [1 << 20, 1 << 24, 1 << 31])
def test_far_positions(fx, far):
    run_case(fx, (64, 4, 64), 64, 0, "half", torch.float32, pos=far - np.arange(64))
    run_case(fx, (64, 4, 64), 64, 0, "interleaved", torch.float32, pos=np.arange(64) - far)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strides(fx, dtype):
    """heads outermost, slices that are not 16-byte aligned, one row repeated, and an output inside a larger one that
    keeps its other values"""
    g = torch.Generator(device="cuda").manual_seed(3)
    big = torch.randn(6, 40, 200, device="cuda", generator=g).to(dtype)
    for x in (big.transpose(0, 1)[:, :, :64], big[:, :, 3:131], big[:, ::3, 8:72], big[:1, :, :64].expand(6, 40, 64)):
        for layout in ("half", "interleaved"):
            buf = torch.full((x.shape[0], x.shape[1] + 1, x.shape[2] + 8), 5.0, dtype=dtype, device="cuda")
            out = buf[:, :-1, :-8]
            run_case(fx, tuple(x.shape), 32, 16, layout, dtype, x=x, out=out)
            assert (buf[:, -1] == 5.0).all() and (buf[:, :, -8:] == 5.0).all()
    y = big.clone()
    run_case(fx, (6, 40, 64), 32, 0, "half", dtype, x=y[:, :, 8:72], in_place=True)
    assert torch.equal(y[:, :, :8], big[:, :, :8]) and torch.equal(y[:, :, 72:], big[:, :, 72:])


def test_outputs_with_heads_outermost(fx):
    for gap in (0, 24):
        buf = torch.full((40, 6 * (64 + gap) + 5), 5.0, device="cuda")
        out = buf.as_strided((6, 40, 64), (64 + gap, buf.stride(0), 1))
        run_case(fx, (6, 40, 64), 32, 16, "half", torch.float32, out=out)
        assert (buf[:, 6 * (64 + gap):] == 5.0).all()


def test_gradient_is_the_inverse_and_matches_differences(fx):
    """y is linear in x: (f(x + d) - f(x)) . w = d . grad, and rotating back gives x again"""
    g = torch.Generator(device="cuda").manual_seed(4)
    x, d, w = (torch.randn(7, 3, 48, device="cuda", generator=g) for _ in range(3))
    freq, ms = fx.rope_freqs(32, scaling="yarn", factor=8.0, original=256.0)
    pos = torch.arange(100, 107, device="cuda")
    for layout in ("half", "interleaved"):
        f = lambda v, inv=False, m=ms: fx.idx_rope(v, pos, freq, offset=5, layout=layout, mscale=m, inverse=inv)
        diff = ((f(x + d).double() - f(x).double()) * w.double()).sum()
        grad = (d.double() * f(w, True).double()).sum()
        # 7 * 3 * 48 terms, each within 2^-20 of values below 4 * 4
        assert abs(float(diff - grad)) <= 7 * 3 * 48 * 2.0 ** -20 * 16
        assert (f(f(x), True, 1.0 / ms) - x).abs().max() <= 2.0 ** -19 * 8


def test_no_tokens_and_a_replayed_graph(fx):
    freq, _ = fx.rope_freqs(64)
    none = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    assert fx.idx_rope(none, torch.empty(0, dtype=torch.int64, device="cuda"), freq).shape == (0, 4, 64)
    x = torch.randn(50, 4, 128, device="cuda").bfloat16()
    pos = torch.arange(50, device="cuda")
    want = fx.idx_rope(x, pos, freq)
    out = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fx.idx_rope(x, pos, freq, out=out)
    for rep in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), rep
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out.zero_()
    torch.cuda.synchronize()
    fx.idx_rope(x, pos, freq, out=out, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
