"""The append with rotation into the 8-bit formats, against the 64-bit oracle bit for bit: tokens whose position has no row in
the table, anywhere in a block."""
import numpy as np
import pytest

from oracle import kv, kv4
from tests.test_gpu_kv4 import _ints, _mbd, _table, dev  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

INT8, E4M3 = kv.INT8, kv.E4M3
ROWS = 300                                                       # of the table


def _steps(dev, fmt, dtype, heads, hq, dim, bs, calls, rot, pairs, unstored, seed=0):  # noqa: F811
    """Appends `calls` (new tokens of each request), each checked whole: codes, scales, turned queries.  The cache holds any codes
    and scales that mean nothing before; unstored(rng, request, position) says whose position has no row."""
    mbd = _mbd()
    rng = np.random.default_rng(seed)
    n = len(calls[0])
    held = -(-np.sum(calls, 0) // bs)
    blocks = int(held.sum()) + 2
    order = rng.permutation(blocks)
    table = np.split(order, np.cumsum(held))[:n]
    codes = [rng.integers(0, 256, (blocks, heads, bs, dim)).astype(np.uint8) for _ in range(2)]
    scales = [np.full((blocks, heads), s, np.float32) for s in (3e30, np.nan)]
    t = lambda a: torch.from_numpy(a.copy()).to(dev)
    cache = mbd.KvCache(mbd.MBD_KV_INT8 if fmt == INT8 else mbd.MBD_KV_E4M3, bs, dim, t(kv.pack(codes[0], False)), t(kv.pack(codes[1], True)),
                        t(scales[0]), t(scales[1]))
    angles = _table(rng, ROWS, rot)
    lens, named = np.zeros(n, int), np.zeros(blocks, int)
    for new in calls:
        at = [(i, p) for i in range(n) for p in range(lens[i], lens[i] + new[i])]
        slots = np.array([table[i][p // bs] * bs + p % bs for i, p in at])
        bad = np.array([unstored(rng, i, p) for i, p in at])
        pos = np.where(bad, rng.choice([-1, ROWS, 2 ** 31 - 1, -2 ** 31], len(at)), rng.integers(0, ROWS, len(at)))
        T, row, qrow = len(at), heads * dim, hq * dim
        x = torch.from_numpy(rng.standard_normal((T, qrow + 2 * row)) * rng.choice([0.3, 1.0, 3.0], (T, 1)))
        x[torch.from_numpy(bad)] *= 1e6                          # what is not stored would be the largest by far
        if T > 9:
            x[np.flatnonzero(bad)[-1:], qrow:] = float("nan")
        x = x.to(torch.bfloat16 if dtype == "bf16" else torch.float32)
        d = x.to(dev)
        k, v = d[:, qrow:qrow + row].unflatten(1, (heads, dim)), d[:, qrow + row:].unflatten(1, (heads, dim))
        q, q_out = (d[:, :qrow].unflatten(1, (hq, dim)), torch.full((T, hq, dim), 7.0, dtype=torch.bfloat16, device=dev)) if hq else (None, None)
        mbd.mbd_kv_append_rope(cache, k, v, _ints(slots, dev), _ints(pos, dev), torch.from_numpy(angles).to(dev), q, q_out, interleaved=pairs)
        torch.cuda.synchronize()
        xn = x.double().numpy()
        kv.append(codes[0], scales[0], kv4.turn(xn[:, qrow:qrow + row].reshape(T, heads, dim), angles, pos, pairs), slots, fmt, ~bad)
        kv.append(codes[1], scales[1], xn[:, qrow + row:].reshape(T, heads, dim), slots, fmt, ~bad)
        np.maximum.at(named, slots // bs, slots % bs + 1)
        lens = lens + new
        got = {m: g.cpu().numpy() for m, g in cache.tensors.items()}
        np.testing.assert_array_equal(got["k_scale"], scales[0])
        np.testing.assert_array_equal(got["v_scale"], scales[1])
        gk, gv = kv.unpack(got["k_codes"], bs, dim, False), kv.unpack(got["v_codes"], bs, dim, True)
        for b in range(blocks):                                  # (behind the last place that was named, codes may be any)
            for name, g, want in (("keys", gk, codes[0]), ("values", gv, codes[1])):
                np.testing.assert_array_equal(g[b, :, :named[b]], want[b, :, :named[b]], err_msg="%s of block %d" % (name, b))
            codes[0][b, :, named[b]:], codes[1][b, :, named[b]:] = gk[b, :, named[b]:], gv[b, :, named[b]:]
        if hq:
            want = torch.from_numpy(kv4.turn(xn[:, :qrow].reshape(T, hq, dim), angles, pos, pairs)).float().to(torch.bfloat16)
            want[torch.from_numpy(bad)] = 7.0
            np.testing.assert_array_equal(q_out.cpu().float().numpy(), want.float().numpy())


UNSTORED = {
    "scattered": lambda rng, i, p: rng.random() < 0.3,
    "first of a block": lambda rng, i, p: p % 16 == 0,
    "all but one": lambda rng, i, p: p % 16 != 11,
    "whole blocks": lambda rng, i, p: p // 16 % 2 == 0,
    "a request's": lambda rng, i, p: i == 1,
}
SHAPES = [  # heads, query heads, dim, block size, calls, rotated channels
    (2, 4, 64, 16, [[5, 20, 3], [1, 1, 1], [17, 0, 40]], 64),                  # a wave a run
    (3, 0, 128, 32, [[1, 33, 70], [9, 0, 5]], 128),
    (1, 2, 192, 64, [[70, 3, 1], [1, 90, 64]], 72),
    (2, 2, 256, 16, [[2, 40, 1], [3, 1, 16]], 256),
    (12, 12, 64, 32, [[100, 77, 9], [150, 40, 3]], 64),                        # windows of tokens
    (12, 0, 128, 256, [[300, 10, 1], [100, 120, 255]], 104),
    (16, 0, 192, 16, [[90, 50, 4], [70, 1, 90]], 192),
    (16, 2, 256, 128, [[129, 30, 1], [3, 90, 100]], 256)]


@pytest.mark.parametrize("heads,hq,dim,bs,calls,rot", SHAPES)
@pytest.mark.parametrize("which", sorted(UNSTORED))
@pytest.mark.parametrize("fmt,dtype,pairs", [(INT8, "bf16", False), (E4M3, "f32", True), (INT8, "f32", True), (E4M3, "bf16", False)])
def test_positions_outside_the_table(dev, heads, hq, dim, bs, calls, rot, which, fmt, dtype, pairs):  # noqa: F811
    print("case rope8 unstored", heads, hq, dim, bs, calls, rot, which, fmt, dtype, pairs, flush=True)
    _steps(dev, fmt, dtype, heads, hq, dim, bs, calls, rot, pairs, UNSTORED[which])


@pytest.mark.parametrize("heads,hq,dim,bs,calls,rot", SHAPES + [
    (16, 0, 128, 128, [[256, 100, 5], [128, 28, 250]], 128),                   # whole blocks whose octets take two rounds and more
    (16, 2, 256, 256, [[256, 200, 1], [300, 56, 255]], 200)])
@pytest.mark.parametrize("fmt,dtype,pairs", [(INT8, "bf16", False), (E4M3, "f32", False), (INT8, "f32", True), (E4M3, "bf16", True)])
def test_every_dimension_and_round(dev, heads, hq, dim, bs, calls, rot, fmt, dtype, pairs):  # noqa: F811
    """All positions in the table: runs of a wave and of a workgroup, windows of many, at every head dimension."""
    print("case rope8", heads, hq, dim, bs, calls, rot, fmt, dtype, pairs, flush=True)
    _steps(dev, fmt, dtype, heads, hq, dim, bs, calls, rot, pairs, lambda rng, i, p: False, seed=1)
