"""Definitions in 64 bits of the rows that idx_write_rows stores and idx_read_rows returns (numpy, value by value from the
formulas). Imported by tests only."""
from __future__ import annotations

import numpy as np

import attn_ref

# values of a row, of a scale's group, code bytes
FORMATS = {"main": (512, 16, 256), "local": (512, 32, 512), "key": (128, 32, 64)}
E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])
E4M3 = attn_ref.e4m3(np.arange(127))


def nearest(v, table):
    """(place of the nearest entry of an ascending table to each |v|, a tie to the even place)"""
    a = np.minimum(np.abs(v), table[-1])
    hi = np.clip(np.searchsorted(table, a), 1, len(table) - 1)
    below, above = a - table[hi - 1], table[hi] - a
    return np.where((above < below) | ((above == below) & (hi % 2 == 0)), hi, hi - 1)


def rotate(x, pos, freq, offset, layout, mscale, inverse=False):
    """x [n, dim] with pair i of its part from `offset` on turned by pos [n] * freq[i]"""
    a = np.asarray(pos, np.float64)[:, None] * freq * (-1 if inverse else 1)
    c, s = np.cos(a) * mscale, np.sin(a) * mscale
    h, y = len(freq), x.astype(np.float64).copy()
    i0 = offset + (np.arange(h) if layout == "half" else 2 * np.arange(h))
    i1 = i0 + (h if layout == "half" else 1)
    y[:, i0], y[:, i1] = x[:, i0] * c - x[:, i1] * s, x[:, i1] * c + x[:, i0] * s
    return y


def normalise(x, gamma, eps):
    y = x / np.sqrt((x * x).mean(1, keepdims=True) + eps)
    return y if gamma is None else y * gamma


def transform(y, signs):
    i = np.arange(128)
    odd = np.array([[bin(a & b).count("1") & 1 for b in i] for a in i])
    return ((y * signs) @ (1.0 - 2.0 * odd)).astype(np.float32) * np.float32(2.0 ** -3.5)


def quantise(format, y):
    """codes [n, width] and scale bytes [n, groups] of rows y (64 bits; a key after its transform)"""
    dim, group, width = FORMATS[format]
    g = np.asarray(y, np.float64).reshape(len(y), dim // group, group)
    top = np.abs(g).max(2)
    if format == "main":
        byte = np.minimum(np.searchsorted(6.0 * E4M3, top), 126)
        s = E4M3[byte]
    else:
        lo, hi, most = (-15, 7, 448.0) if format == "local" else (-127, 127, 6.0)
        byte = np.minimum(np.searchsorted(most * 2.0 ** np.arange(lo, hi + 1.0), top), hi - lo) + lo + 127
        s = 2.0 ** (byte - 127.0)
    v = np.divide(g, s[..., None], out=np.zeros_like(g), where=s[..., None] > 0)
    code = nearest(v, E4M3 if format == "local" else E2M1)
    code = code | np.where((v < 0) & (code > 0), 128 if format == "local" else 8, 0)
    code = code.reshape(len(y), dim).astype(np.uint8)
    if format != "local":
        code = code[:, 0::2] | (code[:, 1::2] << 4)
    return code.reshape(len(y), width), byte.astype(np.uint8)


def values(format, codes, scales):
    """[n, dim] values of stored rows"""
    if format == "main":
        return attn_ref.kv_rows(codes, scales)
    s = 2.0 ** (scales.astype(np.float64) - 127)
    if format == "local":
        v = attn_ref.e4m3(codes)
    else:
        v = attn_ref.E2M1[np.stack([codes & 15, codes >> 4], -1).reshape(len(codes), 128)]
    return v * np.repeat(s, 32, axis=1)


def row_of(i, at, max_n, rows, kv_base=None, pages=None, page_size=0, seq=None, ring=0):
    """Cache row of entry at[i], or -1"""
    p = int(at[i])
    if p < 0 or p >= max_n:
        return -1
    if ring:
        p %= ring
    if pages is not None:
        s = int(seq[i]) if seq is not None else i
        if s < 0 or s >= len(pages) or pages[s][p // page_size] < 0:
            return -1
        r = int(pages[s][p // page_size]) * page_size + p % page_size
    else:
        r = p + (int(kv_base[i]) if kv_base is not None else 0)
    return r if 0 <= r < rows else -1
