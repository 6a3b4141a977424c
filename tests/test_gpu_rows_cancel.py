"""idx_write_rows where a turned value's two products cancel: what is left is small beside the pair it comes from, and so is its
own precision. A code is the nearest to the formula's value but for the error of the 64-bit rotation, 2^-47 of the pair's
magnitudes: the angle 2^-50, sine and cosine 2^-49.8 (the first term left out of the cosine's series, (pi/4)^16 / 16!), two
products and a sum 2^-51, times mscale 2^-53, a norm 2^-48."""
import numpy as np
import pytest
import torch

import rows_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fx():
    import top_fp4_lightning_amd as fx

    return fx


def rows_that_cancel(rng, tokens, layout, mscale, size):
    """(x [tokens, 512] fp32, pos, freq, y, pair): y = what x is turned into, in extended precision, tiny in every first value of
    a pair; pair = |x0| + |x1|"""
    freq = 0.7 * 10000.0 ** (-np.arange(256) / 256)
    pos = rng.integers(1, 200, tokens)
    a = pos.astype(np.longdouble)[:, None] * freq.astype(np.longdouble)
    c, s = np.cos(a), np.sin(a)
    x1 = np.float32(size * (0.5 + rng.random((tokens, 256))))
    x0 = np.float32(x1 * s / c)  # x0 c - x1 s is x0's rounding
    i = np.arange(256)
    i0, i1 = (i, 256 + i) if layout == "half" else (2 * i, 2 * i + 1)
    x, y, pair = np.zeros((tokens, 512), np.float32), np.zeros((tokens, 512), np.longdouble), np.zeros((tokens, 512))
    x[:, i0], x[:, i1] = x0, x1
    y[:, i0], y[:, i1] = (x0 * c - x1 * s) * mscale, (x1 * c + x0 * s) * mscale
    pair[:, i0] = pair[:, i1] = np.abs(x0.astype(np.float64)) + np.abs(x1)
    return x, pos, freq, y, pair


def stored(fx, format, x, pos, freq, layout, mscale):
    dim, group, width = ref.FORMATS[format]
    codes = torch.zeros(len(x), width, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(len(x), dim // group, dtype=torch.uint8, device="cuda")
    dev = lambda v: torch.from_numpy(np.ascontiguousarray(v)).cuda()  # noqa: E731
    fx.idx_write_rows(format, dev(x), codes, scales, torch.arange(len(x), device="cuda"), len(x), pos=dev(pos), freq=dev(freq),
                      layout=layout, mscale=mscale)
    codes, scales = codes.cpu().numpy(), scales.cpu().numpy()
    s = ref.attn_ref.e4m3(scales) if format == "main" else 2.0 ** (scales.astype(np.float64) - 127)
    return ref.values(format, codes, scales), np.repeat(s, group, axis=1), s


def off_by(format, y, got, scale):
    """how much farther than the nearest number of the format the stored one is"""
    table = ref.E4M3 if format == "local" else ref.E2M1
    v = np.abs(y) / scale
    hi = np.clip(np.searchsorted(table, v.astype(np.float64)), 1, len(table) - 1)
    best = np.minimum(np.abs(v - table[hi - 1]), np.abs(v - table[hi])) * scale
    return np.abs(got - y) - best


@pytest.mark.parametrize("format", ["main", "local"])
@pytest.mark.parametrize("layout, mscale, size", [("half", 1.0, 1.0), ("half", 1.25, 2000.0), ("half", 1.0, 2.0 ** 13),
                                                  ("interleaved", 0.75, 30.0)])
def test_cancelling_pairs(fx, format, layout, mscale, size):
    rng = np.random.default_rng(int(size))
    x, pos, freq, y, pair = rows_that_cancel(rng, 1500, layout, mscale, size)
    got, scale, s = stored(fx, format, x, pos, freq, layout, mscale)
    room = 2.0 ** -47 * pair * mscale
    assert (off_by(format, y, got, scale) <= 2 * room).all()
    # the scale: the smallest that holds the group, but for the same error
    dim, group, _ = ref.FORMATS[format]
    top, most = np.abs(y).reshape(len(y), -1, group).max(2), (ref.E4M3 if format == "local" else ref.E2M1)[-1]
    slack = room.reshape(len(y), -1, group).max(2)
    if format == "local":
        largest, smallest, below = s == 2.0 ** 7, s == 2.0 ** -15, s / 2
    else:
        at = np.searchsorted(ref.E4M3, s)
        largest, smallest, below = at == 126, at == 0, ref.E4M3[np.maximum(at - 1, 0)]
    assert ((most * s >= top - slack) | largest).all()
    assert ((most * below < top + slack) | smallest).all()
