"""The 4-bit KV cache and the append with rotation on the GPU against the 64-bit oracles: codes, exponents
and turned queries bit for bit, the read-back, and attention at the lengths, layouts, masks and
memory contents where it can go wrong."""
import numpy as np
import pytest

from oracle import kv, kv4

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

INT8, E4M3 = kv.INT8, kv.E4M3


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import memory_bound_decode_amd as mbd
    mbd.lib()
    return torch.device("cuda:0")


def _mbd():
    import memory_bound_decode_amd as mbd
    return mbd


def _ints(a, dev):
    return torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).to(dev)


class Cache:
    """A device cache full of what memory may hold (any codes, NaN exponents), and its oracle twin."""

    def __init__(self, blocks, heads, dim, bs, dev, seed=0):
        self.rng, self.dev, self.bs, self.dim = np.random.default_rng(seed), dev, bs, dim
        shape = (blocks, heads, bs, dim)
        self.k, self.v = (self.rng.integers(0, 16, shape).astype(np.uint8) for _ in range(2))
        self.ke, self.ve = (np.full(shape[:3] + (dim // 32,), 255, np.uint8) for _ in range(2))

    def fill(self, blocks):
        """Codes of normal values and exponents near 1 in these blocks."""
        for codes, exps in ((self.k, self.ke), (self.v, self.ve)):
            shape = (len(blocks),) + codes.shape[1:]
            codes[blocks] = kv4.encode(self.rng.standard_normal(shape) * 2.2)
            exps[blocks] = self.rng.integers(125, 128, shape[:3] + (self.dim // 32,))

    def spoil(self, block, place):
        """Behind a request's end: whatever was there."""
        for codes, exps in ((self.k, self.ke), (self.v, self.ve)):
            codes[block, :, place:] = self.rng.integers(0, 16, codes[block, :, place:].shape)
            exps[block, :, place:] = 255

    def device(self):
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(self.dev)
        return _mbd().KvCache(_mbd().MBD_KV_MXFP4, self.bs, self.dim, t(kv4.pack(self.k, False)), t(kv4.pack(self.v, True)),
                              t(kv4.pack_scales(self.ke)), t(kv4.pack_scales(self.ve)))

    def check(self, cache):
        got = {k: t.cpu().numpy() for k, t in cache.tensors.items()}
        np.testing.assert_array_equal(kv4.unpack_scales(got["k_scale"], self.bs, self.dim), self.ke)
        np.testing.assert_array_equal(kv4.unpack_scales(got["v_scale"], self.bs, self.dim), self.ve)
        np.testing.assert_array_equal(kv4.unpack(got["k_codes"], self.bs, self.dim, False), self.k)
        np.testing.assert_array_equal(kv4.unpack(got["v_codes"], self.bs, self.dim, True), self.v)

    def values(self, blocks=slice(None)):
        """Values of live memory; what stands behind an exponent of 255 is not read."""
        one = lambda c, e: kv4.values(c[blocks], np.where(e[blocks] == 255, 27, e[blocks]))
        return one(self.k, self.ke), one(self.v, self.ve)


def _table(rng, rows, rot):
    angle = rng.uniform(0, 7, (rows, rot // 2))
    return np.float32(np.concatenate([np.cos(angle), np.sin(angle)], 1))


# ------------------------------------------------------------------ append and gather

APPENDS = [  # blocks, heads, dim, bs, tokens, rotated channels, query heads
    (4, 1, 64, 16, 1, 64, 1), (5, 3, 128, 16, 37, 128, 12), (3, 2, 192, 32, 70, 64, 2), (2, 2, 256, 256, 300, 256, 6), (9, 5, 64, 64, 111, 24, 5),
    (4, 1, 192, 128, 17, 192, 7), (40, 7, 128, 16, 500, 0, 0), (3, 2, 256, 32, 33, 8, 0), (6, 4, 64, 32, 150, 0, 0), (2, 1, 192, 16, 16, 136, 3)]


@pytest.mark.parametrize("blocks,heads,dim,bs,T,rot,hq", APPENDS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pairs", [False, True])
def test_append_and_gather(dev, blocks, heads, dim, bs, T, rot, hq, dtype, pairs):
    """Slots in any order, rows that go nowhere, positions outside the table; special values, slices of a projection."""
    mbd = _mbd()
    print("case append4", blocks, heads, dim, bs, T, rot, hq, dtype, pairs, flush=True)
    c = Cache(blocks, heads, dim, bs, dev, seed=T)
    cache, rng = c.device(), c.rng
    slots = rng.permutation(blocks * bs)[:T]
    if T > 30:
        slots[:20] = np.sort(slots[:20])
    slots = np.concatenate([slots, [-1, blocks * bs, -2 ** 31, 2 ** 31 - 1]])
    T = len(slots)
    rows = 50
    pos = rng.integers(0, rows, T)
    pos[rng.random(T) < 0.1] = rng.choice([-1, rows, 2 ** 31 - 1, -2 ** 31])
    row, qrow = heads * dim, hq * dim
    x = torch.from_numpy(rng.standard_normal((T, qrow + 2 * row + 8)) * rng.choice([1e-30, 0.02, 1.0, 3.0, 1e4], (T, 1)))
    x[0, qrow:qrow + 32] = 0
    x[0, qrow + row + 1] = float("inf")
    if T > 5:
        x[1, qrow + 3], x[1, qrow + row + 5], x[1, qrow + row + 40] = float("nan"), float("-inf"), float("nan")
        x[2, qrow + row:qrow + row + 32] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0] * 4) * torch.tensor([1.0, -1.0] * 16)
        x[3, qrow + row:qrow + row + 32] = 3e38
    x = x.to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    d = x.to(dev)
    q, k, v = (d[:, a:b].unflatten(1, (-1, dim)) if b > a else None for a, b in ((0, qrow), (qrow, qrow + row), (qrow + row, qrow + 2 * row)))
    xn = x.double().numpy()
    kn, vn = xn[:, qrow:qrow + row].reshape(T, heads, dim), xn[:, qrow + row:qrow + 2 * row].reshape(T, heads, dim)
    if rot:
        table = _table(rng, rows, rot)
        out_wide = torch.full((T, qrow + 16), 7.0, dtype=torch.bfloat16, device=dev)
        q_out = out_wide[:, :qrow].unflatten(1, (hq, dim)) if hq else None
        mbd.mbd_kv_append_rope(cache, k, v, _ints(slots, dev), _ints(pos, dev), torch.from_numpy(table).to(dev), q, q_out, interleaved=pairs)
        known = (pos >= 0) & (pos < rows)
        kn, use = kv4.turn(kn, table, pos, pairs), np.where(known, slots, -1)
    else:
        mbd.mbd_kv_append(cache, k, v, _ints(slots, dev))
        use = slots
    torch.cuda.synchronize()
    kv4.append(c.k, c.ke, kn, use)
    kv4.append(c.v, c.ve, vn, use)
    c.check(cache)
    if rot and hq:
        want = torch.from_numpy(kv4.turn(xn[:, :qrow].reshape(T, hq, dim), table, pos, pairs)).to(torch.float32).to(torch.bfloat16)
        want[torch.from_numpy(~known)] = 7.0
        np.testing.assert_array_equal(q_out.cpu().float().numpy(), want.float().numpy())
        assert (out_wide[:, qrow:] == 7).all()
    # read everything back, in another order, with rows that name nothing
    live = np.array([s for s in use if 0 <= s < blocks * bs] + [-1, blocks * bs, 2 ** 31 - 1])
    live = rng.permutation(live)
    good = (live >= 0) & (live < blocks * bs)
    for out_dt in (torch.float32, torch.bfloat16):
        ko = torch.full((len(live), heads, dim), 77.0, dtype=out_dt, device=dev)
        vo = torch.full_like(ko, 77.0)
        mbd.mbd_kv_gather(cache, _ints(live, dev), ko, vo)
        torch.cuda.synchronize()
        b, p = live[good] // bs, live[good] % bs
        for o, codes, exps in ((ko, c.k, c.ke), (vo, c.v, c.ve)):
            want = torch.from_numpy(kv4.values(codes[b, :, p], exps[b, :, p])).float().to(out_dt).float().numpy()
            np.testing.assert_array_equal(o.cpu()[torch.from_numpy(good)].float().numpy(), want)
            assert (o.cpu()[torch.from_numpy(~good)] == 77).all()


def test_append_rounds_as_the_definition(dev):
    """Every fp32 near every tie and end of a binade, at small, middling and large scales."""
    mbd = _mbd()
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0])
    near = np.concatenate([np.nextafter(np.float32(mids), np.float32(t)) for t in (0, 9)] + [np.float32(mids), [0.0]])
    rows = []
    for e in (-120, -101, -100, -60, -3, 0, 5, 100, 124, 125):
        with np.errstate(over="ignore"):
            g = np.float32(np.ldexp(near.astype(np.float64), e))
        rows.append(np.resize(g, 32) * np.where(np.arange(32) % 3 == 0, -1, 1))
        rows.append(np.resize(g[g <= 6.5 * 2.0 ** e], 32))
    x = np.resize(np.float32(rows), (16, 2, 64))
    c = Cache(1, 2, 64, 16, dev)
    cache, t = c.device(), torch.from_numpy(x).to(dev)
    mbd.mbd_kv_append(cache, t, t, _ints(np.arange(16), dev))
    torch.cuda.synchronize()
    kv4.append(c.k, c.ke, x, np.arange(16))
    kv4.append(c.v, c.ve, x, np.arange(16))
    c.check(cache)


ROPE8 = [  # heads, dim, bs, first positions, new counts of each call, rotated channels, query heads
    (1, 64, 16, [0], [[1], [1], [17]], 64, 2), (3, 128, 16, [0, 5, 16, 31], [[1, 1, 1, 1], [2, 0, 17, 33]], 128, 6),
    (2, 192, 32, [0, 30, 7], [[5, 5, 5], [40, 1, 0]], 72, 0), (2, 256, 256, [0, 200], [[300, 100], [1, 1]], 256, 3), (4, 64, 64, [0, 63, 1], [[700, 1, 62]], 16, 8)]


@pytest.mark.parametrize("fmt", [INT8, E4M3])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("heads,dim,bs,first,calls,rot,hq", ROPE8)
def test_rope_append_8_bits(dev, fmt, dtype, pairs, heads, dim, bs, first, calls, rot, hq):
    """Turned keys in blocks that share a scale: every call's codes and scales are those of the turned keys."""
    mbd = _mbd()
    print("case rope8", fmt, dtype, pairs, heads, dim, bs, first, calls, rot, hq, flush=True)
    rng = np.random.default_rng(rot)
    lens = np.array(first)
    held = -(-(lens + np.sum(calls, 0)) // bs)
    blocks = int(held.sum()) + 2
    order, table, at = rng.permutation(blocks), [], 0
    for h in held:
        table.append(order[at:at + h])
        at += h
    codes = [np.full((blocks, heads, bs, dim), 3, np.uint8) for _ in range(2)]
    scales = [np.full((blocks, heads), 2.0 ** -7, np.float32) for _ in range(2)]
    t = lambda a: torch.from_numpy(a.copy()).to(dev)
    cache = mbd.KvCache(mbd.MBD_KV_INT8 if fmt == INT8 else mbd.MBD_KV_E4M3, bs, dim, t(kv.pack(codes[0], False)), t(kv.pack(codes[1], True)),
                        t(scales[0]), t(scales[1]))
    angles = _table(rng, 900, rot)
    live = np.zeros(blocks, int)
    for i, p in enumerate(first):
        for j in range(p):
            live[table[i][j // bs]] = j % bs + 1
    for new in calls:
        at = [(i, p) for i in range(len(lens)) for p in range(lens[i], lens[i] + new[i])]
        slots = np.array([table[i][p // bs] * bs + p % bs for i, p in at] + [-1, blocks * bs])
        pos = np.array([p for _, p in at] + [5, 6])
        if lens.max() > 20:                                  # a run that ends early: its last token's position has no row
            slots, pos = np.append(slots, [order[-1] * bs, order[-1] * bs + 1]), np.append(pos, [899, 900])
        T, row, qrow = len(slots), heads * dim, hq * dim
        x = torch.from_numpy(rng.standard_normal((T, qrow + 2 * row)) * rng.choice([0.3, 1.0, 3.0], (T, 1))).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
        x[0, qrow + 3], x[0, qrow + row + 6] = float("nan"), float("inf")
        d = x.to(dev)
        k, v = d[:, qrow:qrow + row].unflatten(1, (heads, dim)), d[:, qrow + row:].unflatten(1, (heads, dim))
        q, q_out = (d[:, :qrow].unflatten(1, (hq, dim)), torch.full((T, hq, dim), 7.0, dtype=torch.bfloat16, device=dev)) if hq else (None, None)
        mbd.mbd_kv_append_rope(cache, k, v, _ints(slots, dev), _ints(pos, dev), torch.from_numpy(angles).to(dev), q, q_out, interleaved=pairs)
        torch.cuda.synchronize()
        xn, use = x.double().numpy(), np.where(pos < 900, slots, -1)
        kv.append(codes[0], scales[0], kv4.turn(xn[:, qrow:qrow + row].reshape(T, heads, dim), angles, pos, pairs), use, fmt)
        kv.append(codes[1], scales[1], xn[:, qrow + row:].reshape(T, heads, dim), use, fmt)
        for s in use:
            if 0 <= s < blocks * bs:
                live[s // bs] = s % bs + 1
        lens = lens + new
        got = {n: g.cpu().numpy() for n, g in cache.tensors.items()}
        np.testing.assert_array_equal(got["k_scale"][live > 0], scales[0][live > 0])
        np.testing.assert_array_equal(got["v_scale"][live > 0], scales[1][live > 0])
        gk, gv = kv.unpack(got["k_codes"], bs, dim, False), kv.unpack(got["v_codes"], bs, dim, True)
        for b in range(blocks):
            np.testing.assert_array_equal(gk[b, :, :live[b]], codes[0][b, :, :live[b]], err_msg="keys of block %d" % b)
            np.testing.assert_array_equal(gv[b, :, :live[b]], codes[1][b, :, :live[b]], err_msg="values of block %d" % b)
        if hq:
            want = torch.from_numpy(kv4.turn(xn[:, :qrow].reshape(T, hq, dim), angles, pos, pairs)).float().to(torch.bfloat16)
            want[torch.from_numpy(pos >= 900)] = 7.0
            np.testing.assert_array_equal(q_out.cpu().float().numpy(), want.float().numpy())


# ------------------------------------------------------------------ attention

def _case(dev, dim, bs, hkv, group, lens, new, *, scale=None, softcap=0.0, window=0, alibi=False, pad=0, holes=(), seed=0, max_new=None, qpad=0,
          qmul=None, edit=None):
    mbd = _mbd()
    lens, new = np.array(lens), np.array(new)
    n, hq = len(lens), hkv * group
    held = -(-lens // bs)
    blocks = int(held.sum()) + 3
    c = Cache(blocks, hkv, dim, bs, dev, seed=seed)
    order, at = c.rng.permutation(blocks), 0
    width = max(1, int(held.max())) + 1
    table = np.full((n, width), -1)
    for i in range(n):
        table[i, :held[i]] = order[at:at + held[i]]
        at += held[i]
    c.fill(order[:at])
    for i in range(n):
        if lens[i] % bs:
            c.spoil(table[i, lens[i] // bs], lens[i] % bs)
    for i, col in holes:
        table[i, col] = c.rng.choice([-1, blocks, -2 ** 31, 2 ** 31 - 1])
    if edit:
        edit(c, table)
    table_dev = table.copy()
    table_dev[table_dev == -1] = c.rng.choice([-1, blocks + 5])
    start = np.concatenate([[0], np.cumsum(new)])
    T = int(start[-1]) + pad
    x = c.rng.standard_normal((T, hq, dim)) * 1.5
    if qmul is not None:
        x *= qmul(c.rng, x.shape)
    qt = torch.from_numpy(x).to(torch.bfloat16)
    q = qt.double().numpy()
    slopes = np.float32(2.0 ** (-8.0 * np.arange(1, hq + 1) / hq)) if alibi else None
    sc = dim ** -0.5 if scale is None else scale
    cache = c.device()
    wide = torch.full((T, hq * dim + qpad), 9.0, dtype=torch.bfloat16, device=dev)
    wide[:, :hq * dim] = qt.flatten(1).to(dev)
    out_wide = torch.full((T, hq * dim + qpad), 7.0, dtype=torch.bfloat16, device=dev)
    qd, out = (w[:, :hq * dim].unflatten(1, (hq, dim)) for w in (wide, out_wide))
    lse = torch.full((T, hq), 7.0, device=dev)
    most = max(1, int(new.max())) if max_new is None else max_new
    size = mbd.mbd_kv_attn_workspace_bytes(cache, hq, n, most, width)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=dev) if size else None
    dargs = (cache, qd, _ints(start, dev), _ints(lens, dev), _ints(table_dev, dev), out, ws)
    sl = None if slopes is None else torch.from_numpy(slopes).to(dev)
    call = lambda s=None: mbd.mbd_kv_attn(*dargs, max_new=most, scale=sc, softcap=softcap, window=window, slopes=sl, lse=lse, stream=s)
    kd, vd = c.values()
    one = np.ones(kd.shape[:2])
    args = [q, start, lens, table, kd, vd, one, one, bs, sc, softcap, window, slopes]
    ref, ref_lse, mine = kv.attention(*args)
    args[5] = np.abs(vd)
    weight, _, _ = kv.attention(*args)
    for i in range(n):
        mine[start[i] + most:start[i + 1]] = False
    # du, the error of a score: codes under their exponents and bf16 are exact; fp32 sums of dim products, the factors
    # behind them, the cap's exponential, the bias.
    kmax = np.repeat(np.abs(kd).max((0, 2)), group, 0)[None]
    U = abs(sc) * (np.abs(q) * kmax).sum(-1).max() if T else 0.0
    du = 2.0 ** -23 * (dim * U + 8 * U)
    if softcap:
        du += 2.0 ** -20 * softcap
    if slopes is not None:
        du += 2.0 ** -21 * float(np.max(slopes)) * max(int(max(lens)), 1)
    # A weight is off by du and its rounding to bf16, so o by (2 du + 2^-8 + sums) * sum_j w_j |v_j|, and by half a step of bf16 of itself.
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 * 1.01 + 2 * du + (int(lens.max()) / 16 + 64) * 2.0 ** -24) * weight + 1e-30

    def check(tag="", rows=slice(None)):
        o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
        assert (o[~mine] == 7).all() and (l[~mine] == 7).all(), tag
        if qpad:
            assert (out_wide[:, hq * dim:] == 7).all(), tag
        m = np.zeros_like(mine)
        m[rows] = mine[rows]
        assert np.isfinite(o[m]).all(), tag
        off = (np.abs(o - ref) - tol)[m]
        assert (off <= 0).all(), "%s worst %.3g over its tolerance, at %s" % (tag, off.max(), np.unravel_index(off.argmax(), off.shape))
        empty = np.isneginf(ref_lse) & m[:, None]
        assert np.isneginf(l[empty]).all() and (o[empty] == 0).all(), tag
        some = m[:, None] & ~empty
        np.testing.assert_allclose(l[some], ref_lse[some], atol=du + 2.0 ** -19, rtol=2.0 ** -21, err_msg=tag)
    return call, check, dict(out=out_wide, lse=lse, ws=ws, q=wide, cache=cache, c=c)


def _run(dev, *a, **kw):
    print("case attn4", a, {k: v for k, v in kw.items() if k not in ("qmul", "edit")}, flush=True)
    call, check, _ = _case(dev, *a, **kw)
    call()
    torch.cuda.synchronize()
    check()


LENGTHS = [[1], [15], [16], [17], [32], [33], [127], [128], [129], [640], [2, 1000, 64, 31, 1, 513]]


@pytest.mark.parametrize("dim", [64, 128, 192])
@pytest.mark.parametrize("lens", LENGTHS)
def test_attn_lengths(dev, dim, lens):
    _run(dev, dim, 16, 2, 4, lens, [1] * len(lens))


@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("hkv,group", [(1, 1), (3, 1), (1, 8), (2, 16), (1, 17), (1, 40), (1, 71)])
def test_attn_heads_and_dims(dev, dim, hkv, group):
    _run(dev, dim, 32, hkv, group, [70, 200], [1, 1], pad=1)


@pytest.mark.parametrize("bs", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("dim", [64, 256])
def test_attn_block_sizes(dev, bs, dim):
    _run(dev, dim, bs, 2, 3, [bs - 1, bs, bs + 1, 3 * bs + 5], [1, 1, 1, 1])


@pytest.mark.parametrize("new", [[5, 5, 5], [1, 16, 7], [0, 3, 0], [2, 0, 9]])
@pytest.mark.parametrize("dim,group", [(128, 4), (64, 1), (256, 3), (192, 8)])
def test_attn_verify(dev, new, dim, group):
    _run(dev, dim, 16, 2, group, [max(37, new[0]), 300, 1100], new, pad=2, qpad=16)


@pytest.mark.parametrize("dim", [64, 128, 192, 256])
def test_attn_prompts(dev, dim):
    _run(dev, dim, 64, 1, 3, [150, 90], [150, 41], pad=1)


@pytest.mark.parametrize("opts", [dict(softcap=5.0), dict(window=1), dict(window=16), dict(window=100), dict(window=5000), dict(alibi=True),
                                  dict(softcap=20.0, window=70, alibi=True), dict(scale=0.0), dict(scale=-0.0), dict(scale=-0.3), dict(softcap=0.5, scale=3.0),
                                  dict(scale=1e-35), dict(scale=-0.2, softcap=3.0)])
@pytest.mark.parametrize("dim,new", [(128, [1, 1, 1]), (64, [5, 3, 16]), (256, [40, 2, 9]), (192, [1, 2, 3])])
def test_attn_masks_and_biases(dev, opts, dim, new):
    _run(dev, dim, 16, 2, 2, [40, 333, 1500], new, **opts)


def test_attn_empty_rows(dev):
    """Requests with nothing cached, or less than they bring: rows that see no token; a
    request past max_new; requests whose blocks are all left out, or some."""
    for dim in (64, 128, 192):
        _run(dev, dim, 16, 1, 2, [0, 3, 50], [1, 5, 2])
        _run(dev, dim, 16, 1, 2, [0], [3], window=4)
        _run(dev, dim, 16, 2, 2, [40, 30, 64], [4, 2, 7], max_new=3)
        _run(dev, dim, 16, 1, 2, [64, 700, 20], [1, 2, 1], holes=[(0, 1), (1, 0), (1, 7), (1, 43), (2, 0), (2, 1)])


@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("opts", [{}, dict(softcap=8.0, alibi=True), dict(window=300)])
def test_attn_whole_requests(dev, dim, opts):
    """Tables or windows so short that a workgroup takes a whole request: few and many of them, empty ones, all rows of a tile."""
    for hkv, group, lens, new in ((2, 4, [2048, 1, 0, 333, 16], [1, 1, 1, 4, 2]), (1, 3, [700, 40, 0], [5, 0, 3]), (70, 1, [60, 33, 90, 1, 250, 17, 18, 100], [1] * 8)):
        _run(dev, dim, 32, hkv, group, lens, new, pad=1, qpad=8, **opts)
    _run(dev, dim, 16, 1, 2, [5000, 4100], [2, 1], window=1900)


def test_attn_split_long(dev):
    """Long requests beside short ones: parts joined from the workspace."""
    _run(dev, 128, 64, 1, 8, [20000, 1, 300, 4097], [1, 1, 1, 1])
    _run(dev, 64, 16, 2, 2, [6001, 50], [5, 2], softcap=30.0, window=4000)


def test_attn_prompts_beside_decodes(dev):
    """One call with prompt slices, verify steps and single tokens of long contexts."""
    _run(dev, 128, 64, 2, 4, [260, 9000, 33, 5000, 64], [130, 1, 5, 1, 64], pad=2)
    _run(dev, 64, 16, 1, 40, [50, 3000, 3000], [9, 4, 1], window=2500)


def test_attn_row_tiles_beyond_places(dev):
    _run(dev, 256, 32, 4, 16, [9000] + [24] * 70, [1] + [24] * 70)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("opts", [{}, dict(softcap=7.0, alibi=True), dict(window=90), dict(scale=-0.1)])
def test_attn_wide_row_tiles(dev, dim, opts):
    """Prompts of 128 query rows and more: tiles of 64 rows, the last of them with 1 to 64, cut and whole."""
    _run(dev, dim, 16, 1, 1, [700, 300], [128, 65], pad=1, **opts)
    _run(dev, dim, 32, 2, 3, [90, 1000, 50, 0], [60, 43, 1, 22], qpad=8, **opts)
    _run(dev, dim, 64, 1, 4, [9000, 80], [33, 80], **opts)


def test_attn_prompts_beyond_places(dev):
    """More row tiles than places in few requests: the longest start first, and nothing is cut or done twice."""
    _run(dev, 64, 32, 16, 2, [500, 900, 310], [500, 400, 300])
    _run(dev, 64, 32, 16, 2, [310, 4000, 700], [300, 40, 690], window=700)


@pytest.mark.parametrize("n", [5, 33, 40, 63, 64, 65])
def test_attn_shares_of_ragged_requests(dev, n):
    """Requests of all lengths around the chunk that they are cut by, up to and past a wave's lanes."""
    rng = np.random.default_rng(n)
    for dim, hkv in ((64, 4), (128, 32)):
        _run(dev, dim, 16, hkv, 1, [int(x) for x in 2 ** rng.uniform(0, 11, n)], [1] * n)


@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("hkv,group,new,opts", [(16, 2, 1, {}), (16, 5, 3, {}), (16, 1, 1, dict(softcap=9.0, window=200, alibi=True))])
def test_attn_more_requests_than_places(dev, dim, hkv, group, new, opts):
    """So many requests that one wave works on each part; a long one among them is cut, some see nothing."""
    n = 70
    lens = list(np.random.default_rng(2).integers(new, 100, n))
    lens[1] = 1500
    _run(dev, dim, 16, hkv, group, lens, [i % (new + 1) if i else 0 for i in range(n - 1)] + [new], **opts)


def test_attn_more_heads_than_places(dev):
    _run(dev, 64, 16, 1100, 1, [20, 40, 3], [1, 0, 1])


def test_attn_large_scores(dev):
    """Scores far apart: running maxima that move late, weights that underflow."""
    _run(dev, 128, 16, 1, 4, [900], [3], scale=8.0)


@pytest.mark.parametrize("dim", [64, 128, 192])
def test_attn_queries_of_unlike_channels(dev, dim):
    """Rows whose channels differ by up to 2^20, rows near the ends of bf16's range, rows of zeros."""
    def qmul(rng, shape):
        m = 2.0 ** rng.integers(-20, 1, shape)
        m[0, 0], m[1, 0], m[-1, 1] = 0.0, 2.0 ** -110, 2.0 ** 60
        return m
    # (the row of 2^60 meets keys of zeros alone: see below)
    def edit(c, table):
        c.k[:, 0] &= 8
    _run(dev, dim, 16, 1, 2, [70, 200], [2, 1], qmul=qmul, edit=edit)
    _run(dev, dim, 16, 2, 2, [70, 200], [2, 1], qmul=lambda rng, s: 2.0 ** rng.integers(-20, 1, s))


@pytest.mark.parametrize("low,high", [(70, 90), (100, 140), (120, 150)])
def test_attn_exponents_over_their_range(dev, low, high):
    """Exponent bytes far apart within a token, keys and values."""
    def edit(c, table):
        for e in (c.ke, c.ve):
            live = e < 255
            e[live] = c.rng.integers(low, high, live.sum())
    _run(dev, 128, 16, 2, 2, [70, 300], [2, 1], edit=edit, scale=128 ** -0.5 * 2.0 ** (127 - high))


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("dim,new", [(64, 1), (128, 9), (192, 1)])
def test_bad_queries_stay_in_their_row(dev, bad, dim, new):
    call, check, t = _case(dev, dim, 16, 2, 2, [90, 300], [new, new])
    t["q"][1, 3 * dim + 5] = bad
    call()
    torch.cuda.synchronize()
    check(rows=[i for i in range(2 * new) if i != 1])
    o = t["out"][1].unflatten(0, (4, dim))
    assert torch.isnan(o[3].float()).all() and torch.isfinite(o[:3].float()).all()


def test_every_cached_position_counts_once(dev):
    """Keys of zeros: every weight is the same, and the sum of one value channel at each position in turn."""
    mbd = _mbd()
    for dim, bs, length in ((64, 16, 77), (128, 32, 130), (192, 16, 50)):
        hits = np.zeros((length, dim))
        c = Cache(length // bs + 2, 1, dim, bs, dev)
        order = c.rng.permutation(len(c.k))
        c.k[:], c.ke[:], c.ve[:], c.v[:] = 0, 127, 127, 0
        cache = c.device()
        lens, start = _ints([length], dev), _ints([0, 1], dev)
        table = _ints(order[None, :length // bs + 1], dev)
        q, out = torch.ones((1, 1, dim), dtype=torch.bfloat16, device=dev), torch.zeros((1, 1, dim), dtype=torch.bfloat16, device=dev)
        ws = torch.empty(max(16, mbd.mbd_kv_attn_workspace_bytes(cache, 1, 1, 1, table.shape[1])), dtype=torch.uint8, device=dev)
        for p in range(length):
            c.v[:] = 0
            c.v[order[p // bs], :, p % bs] = np.arange(dim) % 7 + 1
            cache.tensors["v_codes"].copy_(torch.from_numpy(kv4.pack(c.v, True)).to(dev))
            mbd.mbd_kv_attn(cache, q, start, lens, table, out, ws)
            hits[p] = out[0, 0].double().cpu().numpy()
        want = kv4.VALUES[np.arange(dim) % 7 + 1] / length
        assert (np.abs(hits - want) <= 2.0 ** -7 * want).all()     # bf16 of the weight and of the output, 2^-8 each


def test_offsets_past_32_bits(dev):
    """Blocks whose byte offsets pass 2^32: a cache of 5 GB, of which a few blocks are used."""
    mbd = _mbd()
    hkv, dim, bs = 8, 256, 256
    blocks = 5 * (1 << 30) // (hkv * dim * bs // 2)
    codes = [torch.empty((blocks, hkv, bs * dim // 2), dtype=torch.uint8, device=dev) for _ in range(2)]
    scales = [torch.empty((blocks, hkv, bs * dim // 32), dtype=torch.uint8, device=dev) for _ in range(2)]
    cache = mbd.KvCache(mbd.MBD_KV_MXFP4, bs, dim, *codes, *scales)
    rng = np.random.default_rng(4)
    table, lens = np.array([[blocks - 1, 0], [blocks - 2, blocks - 3]]), np.array([300, 400])
    slots = np.concatenate([[table[i][p // bs] * bs + p % bs for p in range(lens[i])] for i in range(2)])
    x = torch.from_numpy(rng.standard_normal((700, hkv, 2, dim))).to(torch.bfloat16)
    mbd.mbd_kv_append(cache, x[:, :, 0].contiguous().to(dev), x[:, :, 1].contiguous().to(dev), _ints(slots, dev))
    ko, vo = torch.empty((700, hkv, dim), device=dev), torch.empty((700, hkv, dim), device=dev)
    mbd.mbd_kv_gather(cache, _ints(slots, dev), ko, vo)
    q = torch.from_numpy(rng.standard_normal((2, hkv, dim))).to(torch.bfloat16).to(dev)
    out = torch.zeros_like(q)
    ws = torch.empty(max(16, mbd.mbd_kv_attn_workspace_bytes(cache, hkv, 2, 1, 2)), dtype=torch.uint8, device=dev)
    mbd.mbd_kv_attn(cache, q, _ints([0, 1, 2], dev), _ints(lens, dev), _ints(table, dev), out, ws)
    torch.cuda.synchronize()
    xn = x.double().numpy()
    for o, j in ((ko, 0), (vo, 1)):
        np.testing.assert_array_equal(o.cpu().double().numpy(), kv4.values(*kv4.quantise(xn[:, :, j])))
    k, v, qf = ko.double().cpu(), vo.double().cpu(), q.double().cpu()
    for i, (a, b) in enumerate(((0, 300), (300, 700))):
        w = torch.softmax((k[a:b] * qf[i]).sum(-1).T * dim ** -0.5, 1)
        ref, mag = (w.T[..., None] * v[a:b]).sum(0), (w.T[..., None] * v[a:b].abs()).sum(0)
        assert ((out[i].double().cpu() - ref).abs() <= 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -13) * mag).all()


# ------------------------------------------------------------------ streams, graphs, a step

def test_attn_other_stream_and_graph(dev):
    call, check, t = _case(dev, 128, 16, 2, 4, [700, 3, 90], [2, 1, 5])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(side.cuda_stream)
    side.synchronize()
    check("side stream")
    want = t["out"].clone(), t["lse"].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(None)
    for i in range(3):
        t["out"].fill_(7.0)
        t["lse"].fill_(7.0)
        if t["ws"] is not None:
            t["ws"].fill_(0xFF)                           # eager work between replays
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(t["out"], want[0]) and torch.equal(t["lse"], want[1]), "replay %d" % i


def _formats(mbd):
    return {"mxfp4": mbd.MBD_KV_MXFP4, "int8": mbd.MBD_KV_INT8, "e4m3": mbd.MBD_KV_E4M3}


@pytest.mark.parametrize("fmt", ["mxfp4", "int8", "e4m3"])
@pytest.mark.parametrize("T", [40, 1500])                 # few tokens; so many that windows take them
def test_append_and_gather_on_other_streams_and_in_graphs(dev, fmt, T):
    """Two captured steps over caches of their own, replayed in turn among eager work, against an eager call."""
    mbd = _mbd()
    rng = np.random.default_rng(T)
    heads, hq, dim, bs, blocks = 3, 6, 128, 32, T // 32 + 2
    x = torch.from_numpy(rng.standard_normal((2, T, hq + 2 * heads, dim))).to(torch.bfloat16).to(dev)
    table = torch.from_numpy(_table(rng, T, dim)).to(dev)
    slots, pos = _ints(rng.permutation(blocks - 1)[:, None] * bs + np.arange(bs), dev).flatten()[:T].contiguous(), _ints(np.arange(T), dev)

    def fresh():
        c = mbd.KvCache.empty(_formats(mbd)[fmt], blocks, heads, dim, bs)
        qkv = torch.zeros_like(x[0])
        return c, qkv, torch.zeros((T, hq, dim), dtype=torch.bfloat16, device=dev), torch.zeros((T, heads, dim), device=dev), torch.zeros((T, heads, dim), device=dev)

    def clear(t):
        for s in t[0].tensors.values():
            s.fill_(1)
        for s in t[2:]:
            s.fill_(7.0)

    def step(t, s=None):
        c, qkv, q_out, ko, vo = t
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + heads], qkv[:, hq + heads:]
        mbd.mbd_kv_append_rope(c, k, v, slots, pos, table, q, q_out, stream=s)
        mbd.mbd_kv_gather(c, slots, ko, vo, stream=s)

    def result(t):
        return [a.clone() for a in (*t[2:], *t[0].tensors.values())]

    sets, want = [fresh() for _ in range(2)], []
    for i in range(2):
        clear(sets[0])
        sets[0][1].copy_(x[i])
        step(sets[0])
        torch.cuda.synchronize()
        want.append(result(sets[0]))
    assert not torch.equal(want[0][0], want[1][0])
    side = torch.cuda.Stream()
    clear(sets[1])
    sets[1][1].copy_(x[1])
    side.wait_stream(torch.cuda.current_stream())
    step(sets[1], side.cuda_stream)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(result(sets[1]), want[1]))
    graphs = []
    for t in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(t)
        graphs.append(g)
    for turn in range(3):
        for i, (t, g) in enumerate(zip(sets, graphs)):
            clear(t)
            t[1].copy_(x[(i + turn) % 2])
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for i, t in enumerate(sets):
            assert all(torch.equal(a, b) for a, b in zip(result(t), want[(i + turn) % 2])), "replay %d of graph %d" % (turn, i)


@pytest.mark.parametrize("fmt", ["mxfp4", "int8"])
def test_more_windows_than_a_launch_has_rows(dev, fmt):
    """One call for 4.3 million tokens is what calls for 2^18 each are, written and read back."""
    mbd = _mbd()
    T, dim, bs, piece = 4_300_000, 64, 256, 1 << 18
    blocks = -(-T // bs)
    gen = torch.Generator(device=dev).manual_seed(5)
    x = torch.randn((T, 3, dim), generator=gen, device=dev, dtype=torch.bfloat16)
    q, k, v = x[:, :1], x[:, 1:2], x[:, 2:]
    rng = np.random.default_rng(6)
    table = torch.from_numpy(_table(rng, 1000, dim)).to(dev)
    ids = torch.arange(T, device=dev, dtype=torch.int32)
    slots, pos = blocks * bs - (ids // bs + 1) * bs + ids % bs, (ids % 1003 - 1).contiguous()       # blocks from the last to the first; some positions have no row
    if fmt == "int8":
        pos.clamp_(0, 999)                                # (there a block's tokens stand next to each other)
    got = []
    for pieces in ([(0, T)], [(a, min(a + piece, T)) for a in range(0, T, piece)]):
        c = mbd.KvCache.empty(_formats(mbd)[fmt], blocks, 1, dim, bs)
        for t in c.tensors.values():
            t.fill_(1)
        q_out, ko, vo = (torch.full((T, 1, dim), 7.0, device=dev, dtype=torch.bfloat16) for _ in range(3))
        for a, b in pieces:
            mbd.mbd_kv_append_rope(c, k[a:b], v[a:b], slots[a:b], pos[a:b], table, q[a:b], q_out[a:b])
        for a, b in pieces:
            mbd.mbd_kv_gather(c, slots[a:b], ko[a:b], vo[a:b])
        torch.cuda.synchronize()
        got.append((q_out, ko, vo, *c.tensors.values()))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    known = (pos >= 0) & (pos < 1000)
    assert bool((got[0][0][~known] == 7).all()) and not bool((got[0][0][known] == 7).all(-1).any())
    # and they are the values: 2^-2 of a group's largest apart at most (half a step of a code, a rounding to bf16)
    off = (got[0][2][known].float() - v[known].float()).abs().amax(-1)
    assert bool((off <= v[known].float().abs().amax(-1) * 0.26).all())


def test_attn_repeats_bit_for_bit(dev):
    call, _, t = _case(dev, 128, 32, 4, 4, [5000, 700, 9], [1, 1, 1])
    got = []
    for _ in range(3):
        call()
        torch.cuda.synchronize()
        got.append((t["out"].clone(), t["lse"].clone()))
    assert all(torch.equal(a, got[0][0]) and torch.equal(b, got[0][1]) for a, b in got)


def test_two_streams_with_their_own_workspaces(dev):
    a, b = _case(dev, 128, 16, 1, 4, [3000, 70], [1, 1], seed=1), _case(dev, 64, 16, 2, 2, [2500, 9], [3, 2], seed=2)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        for (call, _, _), s in zip((a, b), streams):
            call(s.cuda_stream)
    torch.cuda.synchronize()
    a[1]("first")
    b[1]("second")


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("dim,rot,pairs", [(64, 64, False), (128, 48, True), (192, 192, False)])
def test_decode_steps(dev, graph, dim, rot, pairs):
    """A run as it is used: prompts, then verify steps of which some tokens are taken back, then an ended
    request whose blocks another takes; slots -> append with rotation -> attention -> an INT4 output
    projection, every step against the oracle on the same inputs."""
    import synth
    from oracle import gemv, int4
    mbd = _mbd()
    rng = np.random.default_rng(11)
    n, hkv, group, bs, width, blocks = 3, 2, 2, 16, 6, 14
    hq, T = hkv * group, 60
    c = Cache(blocks, hkv, dim, bs, dev)
    cache = c.device()
    pool = mbd.KvPool(bs, torch.full((n, width), -1, dtype=torch.int32, device=dev), _ints(np.arange(blocks), dev))
    table, free = np.full((n, width), -1), np.arange(blocks)
    z = lambda s: torch.zeros(s, dtype=torch.int32, device=dev)
    lens, held, n_free, new_dev = z(n), z(n), _ints([blocks], dev), z(n)
    start, slots, pos, status = z(n + 1), z(T), z(T), z(n)
    K = hq * dim
    w = synth.f32_to_bf16_bits((rng.standard_t(4, (128, K)) * 0.02).astype(np.float32))
    proj = mbd.to_device(mbd.mbd_pack(mbd.MBD_INT4_G128, w), dev)
    qw, sw = int4.quantize(w)
    angles = _table(rng, width * bs, rot)
    angles_dev = torch.from_numpy(angles).to(dev)
    qkv = torch.zeros((T, (hq + 2 * hkv) * dim), dtype=torch.bfloat16, device=dev)
    q, k, v = (qkv[:, a * dim:b * dim].unflatten(1, (b - a, dim)) for a, b in ((0, hq), (hq, hq + hkv), (hq + hkv, hq + 2 * hkv)))
    q_turned, out = torch.zeros((T, hq, dim), dtype=torch.bfloat16, device=dev), torch.zeros((T, hq, dim), dtype=torch.bfloat16, device=dev)
    y = torch.zeros((16, 128), device=dev)
    ws = torch.empty(max(16, mbd.mbd_kv_attn_workspace_bytes(cache, hq, n, 50, width)), dtype=torch.uint8, device=dev)

    def step():
        mbd.mbd_kv_slots(pool, new_dev, lens, held, n_free, start, slots, pos, lens, held, n_free, status)
        mbd.mbd_kv_append_rope(cache, k, v, slots, pos, angles_dev, q, q_turned, interleaved=pairs)
        mbd.mbd_kv_attn(cache, q_turned, start, lens, pool.block_table, out, ws, max_new=50)
        mbd.mbd_gemv(proj, out[:16].flatten(1), y)

    g = None
    if graph:
        step()                                          # no request brings anything yet
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        torch.cuda.synchronize()
    r_lens, r_held, r_free = np.zeros(n, int), np.zeros(n, int), blocks
    plan = [([37, 5, 0], [0, 0, 0]), ([4, 4, 10], [2, 0, 0]), ([4, 4, 4], [1, 3, 4]), ([1, -1, 1], [0, 0, 0]), ([1, 50, 1], [0, 0, 0]), ([4, 4, 4], [0, 0, 0])]
    for s, (new, back) in enumerate(plan):
        x = torch.from_numpy(rng.standard_normal(tuple(qkv.shape)) * (0.5 + s)).to(torch.bfloat16)
        qkv.copy_(x)
        new_dev.copy_(_ints(new, dev))
        (g.replay if graph else step)()
        torch.cuda.synchronize()
        ref = kv.slots(new, r_lens, r_held, table, free, r_free, bs, T)
        np.testing.assert_array_equal(slots.cpu().numpy(), ref["slots"])
        np.testing.assert_array_equal(pos.cpu().numpy(), ref["positions"])
        r_lens, r_held, r_free = ref["lens_out"], ref["held_out"], ref["n_free_out"]
        xn = x.double().numpy().reshape(T, -1, dim)
        kv4.append(c.k, c.ke, kv4.turn(xn[:, hq:hq + hkv], angles, ref["positions"], pairs), ref["slots"])
        kv4.append(c.v, c.ve, xn[:, hq + hkv:], ref["slots"])
        c.check(cache)
        qt = torch.from_numpy(kv4.turn(xn[:, :hq], angles, ref["positions"], pairs)).float().to(torch.bfloat16).double().numpy()
        served = ref["positions"] >= 0
        np.testing.assert_array_equal(q_turned.double().cpu().numpy()[served], qt[served])
        kd, vd = c.values()
        one = np.ones(kd.shape[:2])
        args = [qt, ref["seq_start"], r_lens, table, kd, vd, one, one, bs, dim ** -0.5]
        want, _, mine = kv.attention(*args)
        args[5] = np.abs(vd)
        mag, _, _ = kv.attention(*args)
        top = np.abs(qt).max() * np.abs(kd).max() * dim * dim ** -0.5
        du = 2.0 ** -23 * (dim + 8) * top
        o = out.double().cpu().numpy()
        tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -8 * 1.01 + 2 * du + 2.0 ** -17) * mag + 1e-30
        assert (np.abs(o - want) <= tol)[mine & served].all(), "step %d" % s
        obits = out[:16].flatten(1).cpu().view(torch.int16).numpy().view(np.uint16)
        assert gemv.rel_l2(y.cpu().numpy().astype(np.float64), gemv.gemv(int4.dequant(qw, sw), obits)) <= 1e-3
        lens -= _ints(back, dev)                        # drafts that were not accepted
        r_lens = r_lens - np.array(back)


def test_nothing_to_do(dev):
    """No rows, no new tokens: nothing written, nothing launched out of range."""
    mbd = _mbd()
    c = Cache(4, 1, 64, 16, dev)
    cache = c.device()
    empty, none = torch.empty((0, 1, 64), dtype=torch.bfloat16, device=dev), torch.empty(0, dtype=torch.int32, device=dev)
    mbd.mbd_kv_append(cache, empty, empty, none)
    mbd.mbd_kv_append_rope(cache, empty, empty, none, none, torch.zeros((1, 64), device=dev), empty, empty)
    mbd.mbd_kv_gather(cache, none, empty, empty)
    mbd.mbd_kv_attn(cache, empty, _ints([0, 0], dev), _ints([5], dev), _ints([[0]], dev), empty)
    q = torch.zeros((2, 1, 64), dtype=torch.bfloat16, device=dev)
    out = torch.full_like(q, 7.0)
    mbd.mbd_kv_attn(cache, q, _ints([0, 0], dev), _ints([5], dev), _ints([[0]], dev), out)
    torch.cuda.synchronize()
    assert (out == 7).all()
    c.check(cache)


def test_attn_bad_device_data(dev):
    """Starts and lengths that cannot be: taken as within T and the table, nothing out of range."""
    mbd = _mbd()
    c = Cache(8, 1, 64, 16, dev)
    c.fill(np.arange(8))
    cache = c.device()
    q = torch.ones((6, 2, 64), dtype=torch.bfloat16, device=dev)
    for start, lens in (([0, 2 ** 31 - 1, 3], [2 ** 31 - 1, -5]), ([-9, 4, 2], [40, 2 ** 31 - 1]), ([5, 1, 6], [3, 3]), ([-2 ** 31, 0, 6], [-2 ** 31, 17])):
        out = torch.full_like(q, 7.0)
        ws = torch.empty(max(16, mbd.mbd_kv_attn_workspace_bytes(cache, 2, 2, 6, 3)), dtype=torch.uint8, device=dev)
        mbd.mbd_kv_attn(cache, q, _ints(start, dev), _ints(lens, dev), _ints([[0, 1, 2], [3, 4, 5]], dev), out, ws, max_new=6, window=20)
        torch.cuda.synchronize()
        assert torch.isfinite(out.float()).all()
    c.check(cache)
