"""The 8-bit paged KV cache and attention over it, in plain numpy and 64 bits.

Codes are held by (block, head, place, channel), not in the library's tile order; keys_at
and values_at give the byte that the documented layout assigns to a place and channel.
Roundings that are part of a definition (scales are fp32, a code comes from the fp32
quotient) are written out; everything else is float64."""
from __future__ import annotations

import numpy as np

INT8, E4M3 = "int8", "e4m3"


def keys_at(place, d, dim):
    """Byte of (place in block, channel) of a key block with head_dim = dim."""
    tile, t = divmod(place, 16)
    return tile * 16 * dim + (d // 64) * 1024 + (d // 16 % 4) * 256 + t * 16 + d % 16


def values_at(place, d, dim):
    tile, t = divmod(place, 16)
    return tile * 16 * dim + (d // 64) * 1024 + (t // 4) * 256 + (d // 4 % 16) * 16 + d % 4 * 4 + t % 4


def byte_order(block_size, dim, values):
    """[block_size][dim] byte offsets."""
    f = values_at if values else keys_at
    return np.array([[f(p, d, dim) for d in range(dim)] for p in range(block_size)])


def unpack(raw, block_size, dim, values):
    """uint8 [blocks][heads][block_size * dim] -> [blocks][heads][block_size][dim]."""
    return raw[:, :, byte_order(block_size, dim, values)]


def pack(codes, values):
    blocks, heads, bs, dim = codes.shape
    raw = np.empty((blocks, heads, bs * dim), np.uint8)
    raw[:, :, byte_order(bs, dim, values)] = codes
    return raw


def decode(codes, fmt):
    """What a code stands for before scaling."""
    c = codes.astype(np.int64)
    if fmt == INT8:
        return np.where(c > 127, c - 256, c).astype(np.float64)
    e, m = c >> 3 & 15, c & 7
    mag = np.where(e > 0, (8 + m) * 2.0 ** (e - 10), m * 2.0 ** -9)
    mag = np.where((e == 15) & (m == 7), np.nan, mag)
    return np.where(c > 127, -mag, mag)


_E4M3 = decode(np.arange(127), E4M3)          # magnitudes by code, rising


def encode(v, fmt):
    """Codes of scaled values: nearest even, saturating; NaN is 0."""
    v = np.where(np.isnan(v), 0.0, v)
    if fmt == INT8:
        return (np.clip(np.rint(v), -127, 127).astype(np.int64) & 255).astype(np.uint8)
    a = np.minimum(np.abs(v), 448.0)
    hi = np.searchsorted(_E4M3, a).clip(0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _E4M3[lo], _E4M3[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return (code + 128 * np.signbit(v)).astype(np.uint8)


def wanted_scale(amax, fmt):
    if fmt == INT8:
        return np.float32(np.float32(amax) * np.float32(1 / 127))
    if amax == 0:
        return np.float32(0)
    e = -126
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return np.float32(2.0 ** e)


def append(codes, scale, x, slots, fmt):
    """x [T][heads][dim] into codes [blocks][heads][bs][dim] and scale, both updated."""
    blocks, heads, bs, _ = codes.shape
    x = x.astype(np.float64)
    t = 0
    while t < len(slots):
        if not 0 <= slots[t] < blocks * bs:
            t += 1
            continue
        b, fill = divmod(int(slots[t]), bs)
        n = 1
        while t + n < len(slots) and fill + n < bs and slots[t + n] == slots[t] + n:
            n += 1
        for h in range(heads):
            new = x[t:t + n, h]
            fin = np.abs(new[np.isfinite(new)])
            want = wanted_scale(fin.max() if fin.size else 0.0, fmt)
            old = np.float32(scale[b, h]) if fill else np.float32(0)
            now = max(old, want)
            if now > old and fill:
                ratio = np.float64(np.float32(old / now))
                codes[b, h, :fill] = encode(np.float32(decode(codes[b, h, :fill], fmt) * ratio).astype(np.float64), fmt)
            with np.errstate(over="ignore"):
                q = np.float32(new / np.float64(now if now > 0 else 1.0)).astype(np.float64)
            codes[b, h, fill:fill + n] = encode(q, fmt)
            scale[b, h] = now
        t += n


def slots(new, lens, held, table, free, n_free, bs, T):
    """The step's bookkeeping, one request after the other; table and free are updated."""
    n, width = table.shape
    free_cap = len(free)
    bad = [lens[i] < 0 or held[i] < 0 or held[i] > width or lens[i] > held[i] * bs for i in range(n)]
    for i in range(n):
        if new[i] < 0 and not bad[i]:
            for c in range(held[i]):
                if n_free < free_cap:
                    free[n_free] = table[i, c]
                    n_free += 1
    start = [0]
    lens_out, held_out, status = list(lens), list(held), [4 if b else 0 for b in bad]
    slot, pos = np.full(T, -1, np.int64), np.full(T, -1, np.int64)
    asked, top = 0, n_free
    for i in range(n):
        begin, end = start[-1], start[-1] + max(int(new[i]), 0)
        start.append(end)
        if bad[i]:
            continue
        if new[i] < 0:
            lens_out[i] = held_out[i] = 0
            continue
        if new[i] == 0:
            continue
        want = -(-(int(lens[i]) + int(new[i])) // bs)
        if want > width:
            status[i] = 2
            continue
        if end > T:
            status[i] = 3
            continue
        need = max(want - int(held[i]), 0)
        asked += need
        if need and asked > top:
            status[i] = 1
            continue
        for c in range(held[i], held[i] + need):
            n_free -= 1
            table[i, c] = free[n_free]
        held_out[i] = held[i] + need
        lens_out[i] = lens[i] + new[i]
        for j in range(new[i]):
            p = int(lens[i]) + j
            pos[begin + j] = p
            slot[begin + j] = table[i, p // bs] * bs + p % bs
    return dict(seq_start=np.minimum(start, T), slots=slot, positions=pos, lens_out=np.array(lens_out), held_out=np.array(held_out),
                n_free_out=n_free, status=np.array(status))


def attention(q, seq_start, lens, table, k, v, k_scale, v_scale, bs, scale, softcap=0.0, window=0, slopes=None):
    """q [T][heads][dim] float64; k, v decoded codes [blocks][kv heads][bs][dim].  Returns
    (o, lse, row is a query) in float64."""
    T, heads, dim = q.shape
    group = heads // k.shape[1]
    blocks = k.shape[0]
    o, lse, mine = np.zeros((T, heads, dim)), np.full((T, heads), -np.inf), np.zeros(T, bool)
    for i in range(len(lens)):
        a, b = int(seq_start[i]), int(seq_start[i + 1])
        length = int(lens[i])
        j = np.arange(length)
        ids = table[i][j // bs] if length else np.zeros(0, np.int64)
        there = (ids >= 0) & (ids < blocks)
        j, ids = j[there], ids[there]
        for r in range(a, b):
            mine[r] = True
            at = length - (b - a) + r - a
            see = j <= at
            if window:
                see &= at - j < window
            if not see.any():
                continue
            js, bl = j[see], ids[see]
            for h in range(heads):
                kh = k[bl, h // group, js % bs] * k_scale[bl, h // group][:, None].astype(np.float64)
                vh = v[bl, h // group, js % bs] * v_scale[bl, h // group][:, None].astype(np.float64)
                u = scale * (kh @ q[r, h])
                if softcap:
                    u = softcap * np.tanh(u / softcap)
                if slopes is not None:
                    u = u + float(slopes[h]) * (js - at)
                m = u.max()
                p = np.exp(u - m)
                lse[r, h] = m + np.log(p.sum())
                o[r, h] = p @ vh / p.sum()
    return o, lse, mine
