"""The 4-bit KV cache (e2m1 codes, a power of two for each 32 channels of a token) and the rotation of
keys and queries by position, in plain numpy and 64 bits.

Codes are held by (block, head, place, channel) and exponents by (block, head, place, group), not in the
library's tile order; code_at and scale_at give the nibble and the byte that the documented layout assigns.
Roundings that are part of a definition are written out; everything else is float64."""
from __future__ import annotations

import numpy as np

VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BIAS, LOW, HIGH = 127, -100, 125


def code_at(place, d, dim, values):
    """(byte, half) of (place in block, channel) of a block with head_dim = dim."""
    tile, t = divmod(place, 16)
    base = tile * 8 * dim
    if not values:
        return base + (d // 32) * 256 + t * 16 + d % 32 // 2, d % 2
    if d < dim // 128 * 128:
        return base + (d // 128) * 1024 + (t // 4) * 256 + (d % 128 // 8) * 16 + (t % 4) * 4 + d % 8 // 2, d % 2
    return base + (d // 128) * 1024 + (t // 4) * 128 + (d % 64 // 4) * 8 + (t % 4) * 2 + d % 4 // 2, d % 2


def scale_at(place, group, dim):
    tile, t = divmod(place, 16)
    return tile * (dim // 2) + group * 16 + t


def _order(bs, dim, values):
    at = np.array([[code_at(p, d, dim, values) for d in range(dim)] for p in range(bs)])
    return at[..., 0], at[..., 1]


def _scale_order(bs, dim):
    return np.array([[scale_at(p, g, dim) for g in range(dim // 32)] for p in range(bs)])


def unpack(raw, bs, dim, values):
    """uint8 [blocks][heads][bs * dim / 2] -> codes [blocks][heads][bs][dim]."""
    byte, half = _order(bs, dim, values)
    return raw[:, :, byte] >> (4 * half).astype(np.uint8) & 15


def pack(codes, values):
    blocks, heads, bs, dim = codes.shape
    byte, half = _order(bs, dim, values)
    raw = np.zeros((blocks, heads, bs * dim // 2), np.uint8)
    for h in (0, 1):
        raw[:, :, byte[half == h]] |= codes[:, :, half == h] << np.uint8(4 * h)
    return raw


def unpack_scales(raw, bs, dim):
    return raw[:, :, _scale_order(bs, dim)]


def pack_scales(exps):
    blocks, heads, bs, groups = exps.shape
    raw = np.empty((blocks, heads, bs * groups), np.uint8)
    raw[:, :, _scale_order(bs, groups * 32)] = exps
    return raw


def decode(codes):
    return np.where(codes > 7, -1.0, 1.0) * VALUES[codes & 7]


def values(codes, exps):
    """Values of codes [..., dim] under exponent bytes [..., dim / 32]."""
    return decode(codes) * np.repeat(2.0 ** (exps.astype(np.float64) - BIAS), 32, -1)


def exponent(amax):
    """The smallest e from LOW to HIGH with amax <= 7 * 2^e."""
    e = np.full(np.shape(amax), LOW)
    for k in range(LOW, HIGH):
        e = np.where(np.asarray(amax) > 7 * 2.0 ** k, k + 1, e)
    return e


def encode(v):
    """Codes of scaled values: nearest, ties to the even code, saturating; NaN is 0."""
    a = np.minimum(np.abs(np.where(np.isnan(v), 0.0, v)), 6.0)
    hi = np.searchsorted(VALUES, a).clip(0, 7)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - VALUES[lo], VALUES[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return (code + 8 * (np.signbit(v) & ~np.isnan(v))).astype(np.uint8)


def quantise(x):
    """x [..., dim] -> codes, exponent bytes [..., dim / 32]."""
    g = np.asarray(x, np.float64).reshape(*x.shape[:-1], -1, 32)
    e = exponent(np.where(np.isfinite(g), np.abs(g), 0.0).max(-1))
    return encode(g / 2.0 ** e[..., None]).reshape(x.shape), (e + BIAS).astype(np.uint8)


def append(codes, exps, x, slots):
    """x [T][heads][dim] into codes [blocks][heads][bs][dim] and exps, both updated."""
    blocks, _, bs, _ = codes.shape
    for t, s in enumerate(slots):
        if 0 <= s < blocks * bs:
            codes[s // bs, :, s % bs], exps[s // bs, :, s % bs] = quantise(x[t])


def turn(x, table, positions, interleaved=False):
    """x [T][heads][dim] with its first table.shape[1] channels turned; rows of positions outside the table as they are."""
    rot = table.shape[1]
    out = np.array(x, np.float64)
    f = lambda v: np.float32(v).astype(np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        for t, p in enumerate(positions):
            if not 0 <= p < len(table):
                continue
            for j in range(rot // 2):
                ia, ib = (2 * j, 2 * j + 1) if interleaved else (j, j + rot // 2)
                a, b, c, s = out[t, :, ia].copy(), out[t, :, ib].copy(), float(table[p, j]), float(table[p, rot // 2 + j])
                out[t, :, ia] = f(f(a * c) - f(b * s))
                out[t, :, ib] = f(f(b * c) + f(a * s))
    return out
