"""The KV-cache calls on the GPU against the 64-bit oracle: block tables and slot maps,
the 8-bit append (codes and scales bit for bit), the read-back, and attention at the
lengths, layouts, masks and memory contents where it can go wrong."""
import numpy as np
import pytest

from oracle import kv

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


def _fmt(fmt):
    return _mbd().MBD_KV_INT8 if fmt == INT8 else _mbd().MBD_KV_E4M3


def _ints(a, dev):
    return torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).to(dev)


# ------------------------------------------------------------------ slots

def _requests(seed, n, bs, width, prompt_hi=40):
    """Random requests in every state: decoding, prompts, ended, idle, rolled back, impossible."""
    rng = np.random.default_rng(seed)
    held = rng.integers(0, width + 1, n)
    lens = np.array([rng.integers(0, h * bs + 1) for h in held])
    new = rng.choice([0, 1, 1, 1, 5, -1, -3], n)
    prompts = rng.random(n) < 0.15
    new[prompts] = rng.integers(1, prompt_hi + 1, prompts.sum())
    broken = rng.random(n) < 0.05
    lens[broken] = rng.choice([-1, 10 ** 6], broken.sum())
    held_bad = rng.random(n) < 0.03
    held[held_bad] = width + 1
    total = int(np.clip(held, 0, width).sum())
    free = max(1, n // 3)
    pool = rng.permutation(total + free + 3)
    table = np.full((n, width), -1)
    at = 0
    for i in range(n):
        h = min(held[i], width)
        table[i, :h] = pool[at:at + h]
        at += h
    stack = np.full(len(pool), -7)
    stack[:free] = pool[at:at + free]
    return new, lens, held, table, stack, free


SLOT_CASES = [(1, 1, 16, 4), (2, 5, 16, 3), (3, 33, 32, 6), (4, 64, 16, 8), (5, 200, 128, 2), (6, 1023, 16, 3), (7, 1025, 16, 4),
              (8, 4096, 256, 2), (9, 700, 64, 1)]


@pytest.mark.parametrize("seed,n,bs,width", SLOT_CASES)
@pytest.mark.parametrize("room", ["exact", "padded", "short"])
@pytest.mark.parametrize("in_place", [False, True])
def test_slots(dev, seed, n, bs, width, room, in_place):
    mbd = _mbd()
    print("case slots", seed, n, bs, width, room, in_place, flush=True)
    new, lens, held, table, free, n_free = _requests(seed, n, bs, width)
    total = int(np.maximum(new, 0).sum())
    T = {"exact": total, "padded": total + 37, "short": total // 2}[room]
    ref_table, ref_free = table.copy(), free.copy()
    ref = kv.slots(new, lens, held, ref_table, ref_free, n_free, bs, T)
    pool = mbd.KvPool(bs, _ints(table, dev), _ints(free, dev))
    d = {k: _ints(v, dev) for k, v in dict(new=new, lens=lens, held=held, n_free=[n_free]).items()}
    o = {k: torch.full((s,), -55, dtype=torch.int32, device=dev) for k, s in dict(
        seq_start=n + 1, slots=T, positions=T, lens_out=n, held_out=n, n_free_out=1, status=n).items()}
    if in_place:
        o["lens_out"], o["held_out"], o["n_free_out"] = d["lens"], d["held"], d["n_free"]
    mbd.mbd_kv_slots(pool, d["new"], d["lens"], d["held"], d["n_free"], o["seq_start"], o["slots"], o["positions"], o["lens_out"],
                     o["held_out"], o["n_free_out"], o["status"])
    torch.cuda.synchronize()
    for name, want in ref.items():
        np.testing.assert_array_equal(o[name].cpu().numpy(), np.atleast_1d(want), err_msg=name)
    np.testing.assert_array_equal(pool.block_table.cpu().numpy(), ref_table)
    np.testing.assert_array_equal(pool.free_blocks.cpu().numpy(), ref_free)


def test_slots_long_prompts(dev):
    mbd = _mbd()
    n, bs, width = 3, 16, 5000
    table, free = np.full((n, width), -1), np.random.default_rng(0).permutation(9000)
    new, lens, held = np.array([70001, 3, 1]), np.zeros(3, int), np.zeros(3, int)
    ref_table, ref_free = table.copy(), free.copy()
    ref = kv.slots(new, lens, held, ref_table, ref_free, 9000, bs, 70020)
    pool = mbd.KvPool(bs, _ints(table, dev), _ints(free, dev))
    z = lambda s: torch.zeros(s, dtype=torch.int32, device=dev)
    out = [z(n + 1), z(70020), None, z(n), z(n), z(1), z(n)]
    mbd.mbd_kv_slots(pool, _ints(new, dev), _ints(lens, dev), _ints(held, dev), _ints([9000], dev), *out)
    torch.cuda.synchronize()
    for t, name in zip(out, ("seq_start", "slots", None, "lens_out", "held_out", "n_free_out", "status")):
        if t is not None:
            np.testing.assert_array_equal(t.cpu().numpy(), np.atleast_1d(ref[name]), err_msg=name)
    np.testing.assert_array_equal(pool.block_table.cpu().numpy(), ref_table)


def test_slots_bad_device_data(dev):
    """A free count and block ids that cannot be: nothing is read or written out of range,
    and no slot outside the pool comes out."""
    mbd = _mbd()
    pool = mbd.KvPool(16, _ints([[10 ** 8, -5], [1, 2]], dev), _ints([2 * 10 ** 9, -3, 7, 0], dev))
    z = lambda s: torch.zeros(s, dtype=torch.int32, device=dev)
    start, slots, pos, status = z(3), z(40), z(40), z(2)
    mbd.mbd_kv_slots(pool, _ints([9, 3], dev), _ints([10, 29], dev), _ints([1, 2], dev), _ints([10 ** 9], dev), start, slots, pos, z(2), z(2),
                     z(1), status)
    torch.cuda.synchronize()
    s = slots.cpu().numpy()
    assert ((s >= -1) & (s < 64)).all() and start.tolist() == [0, 9, 12]
    assert s[9:12].tolist() == [2 * 16 + 13, 2 * 16 + 14, 2 * 16 + 15]


# ------------------------------------------------------------------ append and gather

class Cache:
    """A device cache full of what memory may hold (NaN codes, NaN scales), and its oracle twin."""

    def __init__(self, fmt, blocks, heads, dim, bs, dev, seed=0):
        rng = np.random.default_rng(seed)
        self.fmt, self.bs, self.dim = fmt, bs, dim
        fill = 0x7F if fmt == E4M3 else 0x80
        self.k = np.full((blocks, heads, bs, dim), fill, np.uint8)
        self.v = self.k.copy()
        self.ks, self.vs = np.full((blocks, heads), np.nan, np.float32), np.full((blocks, heads), np.nan, np.float32)
        self.rng, self.dev = rng, dev

    def fill(self, blocks):
        """Finite random codes and scales in these blocks."""
        shape = (len(blocks),) + self.k.shape[1:]
        for codes, scale in ((self.k, self.ks), (self.v, self.vs)):
            std = 36 if self.fmt == INT8 else 100
            codes[blocks] = kv.encode(self.rng.standard_normal(shape) * std, self.fmt)
            u = self.rng.random((len(blocks), shape[1]))
            scale[blocks] = (2.6 + 1.4 * u) / 127 if self.fmt == INT8 else np.where(u < 0.5, 2.0 ** -7, 2.0 ** -6)

    def device(self):
        t = lambda a: torch.from_numpy(a.copy()).to(self.dev)
        return _mbd().KvCache(_fmt(self.fmt), self.bs, self.dim, t(kv.pack(self.k, False)), t(kv.pack(self.v, True)), t(self.ks), t(self.vs))

    def check(self, cache):
        got = {k: t.cpu().numpy() for k, t in cache.tensors.items()}
        np.testing.assert_array_equal(got["k_scale"], self.ks)
        np.testing.assert_array_equal(got["v_scale"], self.vs)
        np.testing.assert_array_equal(kv.unpack(got["k_codes"], self.bs, self.dim, False), self.k)
        np.testing.assert_array_equal(kv.unpack(got["v_codes"], self.bs, self.dim, True), self.v)


def _live_only(c, live):
    """Codes past a block's live tokens may hold anything: both sides get the same."""
    for b in range(c.k.shape[0]):
        c.k[b, :, live[b]:] = 0
        c.v[b, :, live[b]:] = 0


APPENDS = [  # blocks, heads, dim, bs, first positions, new counts of each call
    (9, 1, 64, 16, [0], [[1], [1], [1], [14], [3]]),
    (20, 3, 128, 16, [0, 5, 16, 31], [[1, 1, 1, 1], [2, 0, 17, 33], [1, 1, 1, 1]]),
    (12, 2, 192, 32, [0, 30, 7], [[5, 5, 5], [5, 5, 5], [40, 1, 0]]),
    (8, 2, 256, 256, [0, 200], [[300, 100], [1, 1]]),
    (10, 5, 64, 64, [0, 63, 1], [[200, 1, 62], [1, 1, 2]]),
    (6, 2, 128, 128, [0, 127], [[128, 2], [70, 3]]),
]


@pytest.mark.parametrize("fmt", [INT8, E4M3])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("blocks,heads,dim,bs,first,calls", APPENDS)
def test_append_and_gather(dev, fmt, dtype, blocks, heads, dim, bs, first, calls):
    mbd = _mbd()
    print("case append", fmt, dtype, blocks, heads, dim, bs, first, calls, flush=True)
    c = Cache(fmt, blocks, heads, dim, bs, dev, seed=blocks)
    order = c.rng.permutation(blocks)
    ends = np.array(first) + np.sum(calls, 0)
    held = -(-ends // bs)
    assert held.sum() <= blocks
    table, at = [], 0
    for h in held:
        table.append(order[at:at + h])
        at += h
    live = np.zeros(blocks, int)
    for i, p in enumerate(first):
        for j in range(p):
            live[table[i][j // bs]] = j % bs + 1
    c.fill(np.flatnonzero(live))
    _live_only(c, live)
    cache = c.device()
    lens = np.array(first)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    for call, new in enumerate(calls):
        slots = [table[i][p // bs] * bs + p % bs for i in range(len(lens)) for p in range(lens[i], lens[i] + new[i])]
        slots = np.array(slots + [-1, blocks * bs, -2 ** 31])                  # rows that go nowhere
        T, row = len(slots), heads * dim
        x = torch.from_numpy(c.rng.standard_normal((T, 2 * row + 8)) * c.rng.choice([0.3, 1.0, 3.0], (T, 1))).to(dt)
        x[0, :2] = 0
        if call == 1:
            x[0, 3], x[0, 4], x[0, row + 5], x[0, row + 6] = float("inf"), float("nan"), float("-inf"), float("nan")
        d = x.to(dev)
        k, v = d[:, :row].unflatten(1, (heads, dim)), d[:, row:2 * row].unflatten(1, (heads, dim))
        mbd.mbd_kv_append(cache, k, v, _ints(slots, dev))
        torch.cuda.synchronize()
        xn = x.double().numpy()
        kv.append(c.k, c.ks, xn[:, :row].reshape(T, heads, dim), slots, fmt)
        kv.append(c.v, c.vs, xn[:, row:2 * row].reshape(T, heads, dim), slots, fmt)
        for s in slots:
            if 0 <= s < blocks * bs:
                live[s // bs] = s % bs + 1
        lens = lens + new
        got = {n: t.cpu().numpy() for n, t in cache.tensors.items()}
        used = live > 0
        np.testing.assert_array_equal(got["k_scale"][used], c.ks[used])
        np.testing.assert_array_equal(got["v_scale"][used], c.vs[used])
        assert np.isnan(got["k_scale"][~used]).all() and np.isnan(got["v_scale"][~used]).all()
        gk, gv = kv.unpack(got["k_codes"], bs, dim, False), kv.unpack(got["v_codes"], bs, dim, True)
        for b in range(blocks):
            np.testing.assert_array_equal(gk[b, :, :live[b]], c.k[b, :, :live[b]], err_msg="keys of block %d, call %d" % (b, call))
            np.testing.assert_array_equal(gv[b, :, :live[b]], c.v[b, :, :live[b]], err_msg="values of block %d, call %d" % (b, call))
        # read everything back, in another order, with rows that name nothing
        read = np.array([b * bs + p for b in range(blocks) for p in range(live[b])] + [-1, blocks * bs, 2 ** 31 - 1])
        read = c.rng.permutation(read)
        for out_dt in (torch.float32, torch.bfloat16):
            ko = torch.full((len(read), heads, dim), 77.0, dtype=out_dt, device=dev)
            vo = torch.full_like(ko, 77.0)
            mbd.mbd_kv_gather(cache, _ints(read, dev), ko, vo)
            torch.cuda.synchronize()
            good = (read >= 0) & (read < blocks * bs)
            for o, codes, scale in ((ko, c.k, c.ks), (vo, c.v, c.vs)):
                b, p = read[good] // bs, read[good] % bs
                want = (kv.decode(codes[b, :, p], fmt) * scale[b][..., None].astype(np.float64)).astype(np.float32)
                np.testing.assert_array_equal(o.cpu()[torch.from_numpy(good)].float().numpy(), torch.from_numpy(want).to(out_dt).float().numpy())
                assert (o.cpu()[torch.from_numpy(~good)] == 77).all()


@pytest.mark.parametrize("fmt", [INT8, E4M3])
def test_append_many_single_tokens(dev, fmt):
    """More single-token runs than waves look at one by one (windows of several tokens)."""
    mbd = _mbd()
    blocks, heads, dim, bs = 5000, 4, 64, 16
    c = Cache(fmt, blocks, heads, dim, bs, dev)
    cache = c.device()
    slots = c.rng.permutation(blocks)[:4500] * bs
    x = torch.from_numpy(c.rng.standard_normal((len(slots), heads, dim))).to(torch.bfloat16)
    mbd.mbd_kv_append(cache, x.to(dev), (2 * x).to(dev), _ints(slots, dev))
    ko, vo = torch.zeros((len(slots), heads, dim), device=dev), torch.zeros((len(slots), heads, dim), device=dev)
    mbd.mbd_kv_gather(cache, _ints(slots, dev), ko, vo)
    torch.cuda.synchronize()
    kv.append(c.k, c.ks, x.double().numpy(), slots, fmt)
    kv.append(c.v, c.vs, 2 * x.double().numpy(), slots, fmt)
    for o, codes, scale in ((ko, c.k, c.ks), (vo, c.v, c.vs)):
        want = kv.decode(codes[slots // bs, :, 0], fmt) * scale[slots // bs][..., None].astype(np.float64)
        np.testing.assert_array_equal(o.cpu().numpy(), want.astype(np.float32))


@pytest.mark.parametrize("fmt", [INT8, E4M3])
def test_append_zeros_and_tiny(dev, fmt):
    """All-zero tokens (scale 0, codes 0), then values, then the smallest that a scale holds."""
    mbd = _mbd()
    c = Cache(fmt, 3, 1, 64, 16, dev)
    cache = c.device()
    for s, mag in ((0, 0.0), (1, 1.0), (16, 1e-37), (17, 0.0), (32, 3e38)):
        x = np.float32(c.rng.uniform(-1, 1, (1, 1, 64)) * mag)
        t = torch.from_numpy(x).to(dev)
        mbd.mbd_kv_append(cache, t, t, _ints([s], dev))
        kv.append(c.k, c.ks, x, [s], fmt)
        kv.append(c.v, c.vs, x, [s], fmt)
    torch.cuda.synchronize()
    got = {n: t.cpu().numpy() for n, t in cache.tensors.items()}
    np.testing.assert_array_equal(got["k_scale"], c.ks)
    np.testing.assert_array_equal(got["v_scale"], c.vs)
    for b, n in ((0, 2), (1, 2), (2, 1)):
        np.testing.assert_array_equal(kv.unpack(got["k_codes"], 16, 64, False)[b, 0, :n], c.k[b, 0, :n])
        np.testing.assert_array_equal(kv.unpack(got["v_codes"], 16, 64, True)[b, 0, :n], c.v[b, 0, :n])


# ------------------------------------------------------------------ attention

def _tolerances(q, c, table, lens, seq_start, bs, group, scale, softcap, slopes, ref, n_max):
    """What the roundings allow, per output (dim axis last), from the operands' magnitudes.
    du: error of a score, from fp32 sums of dim products, of the factors behind them, of
    the cap's exponential and of the bias.  A weight is then off by du + 2^-8 (its rounding
    to bf16) relative, so o is off by at most (2 du + 2^-8 + sums) * sum_j w_j |v_j|, and by
    half a step of bf16 (2^-8) of itself; sums of n terms in fp32 add n * 2^-24."""
    kd, vd = np.abs(np.nan_to_num(kv.decode(c.k, c.fmt))), np.abs(np.nan_to_num(kv.decode(c.v, c.fmt)))
    kmax = (kd.max(2) * np.nan_to_num(c.ks)[..., None]).max(0)              # [kv heads][dim]
    # U bounds |scale| sum |q||k|, a magnitude, so a negative scale enters by its absolute value
    U = abs(scale) * (np.abs(q) * np.repeat(kmax, group, 0)[None]).sum(-1).max()
    du = 2.0 ** -23 * (q.shape[-1] * U + 8 * U)
    if softcap:
        du += 2.0 ** -20 * softcap
    if slopes is not None:
        du += 2.0 ** -21 * float(np.max(slopes)) * max(int(max(lens)), 1)
    return du


def _abs_attention(args, v_abs):
    a = list(args)
    a[5] = v_abs
    return kv.attention(*a)


def _attn_case(dev, fmt, dim, bs, hkv, group, lens, new, *, scale=None, softcap=0.0, window=0, alibi=False, pad=0, holes=(), seed=0, max_new=None,
               qpad=0, stream=None):
    mbd = _mbd()
    lens, new = np.array(lens), np.array(new)
    n, hq = len(lens), hkv * group
    held = -(-lens // bs)
    blocks = int(held.sum()) + 3
    c = Cache(fmt, blocks, hkv, dim, bs, dev, seed=seed)
    order = c.rng.permutation(blocks)
    width = max(1, int(held.max())) + 1
    table = np.full((n, width), -1)
    at = 0
    for i in range(n):
        table[i, :held[i]] = order[at:at + held[i]]
        at += held[i]
    c.fill(order[:at])
    fill = 0x7F if fmt == E4M3 else 0x80
    for i in range(n):                                    # behind a request's end: whatever was there
        if lens[i] % bs:
            b = table[i, lens[i] // bs]
            c.k[b, :, lens[i] % bs:] = fill
            c.v[b, :, lens[i] % bs:] = fill
    for i, col in holes:
        table[i, col] = c.rng.choice([-1, blocks, -2 ** 31, 2 ** 31 - 1])
    table_dev = table.copy()
    table_dev[table_dev == -1] = c.rng.choice([-1, blocks + 5])
    start = np.concatenate([[0], np.cumsum(new)])
    T = int(start[-1]) + pad
    qt = torch.from_numpy(c.rng.standard_normal((T, hq, dim)) * 1.5).to(torch.bfloat16)
    q = qt.double().numpy()
    slopes = np.float32(2.0 ** (-8.0 * np.arange(1, hq + 1) / hq)) if alibi else None
    sc = dim ** -0.5 if scale is None else scale
    cache = c.device()
    wide = torch.full((T, hq * dim + qpad), 9.0, dtype=torch.bfloat16, device=dev)
    wide[:, :hq * dim] = qt.flatten(1).to(dev)
    qd = wide[:, :hq * dim].unflatten(1, (hq, dim))
    out_wide = torch.full((T, hq * dim + qpad), 7.0, dtype=torch.bfloat16, device=dev)
    out = out_wide[:, :hq * dim].unflatten(1, (hq, dim))
    lse = torch.full((T, hq), 7.0, device=dev)
    most = int(new.max()) if max_new is None else max_new
    size = mbd.mbd_kv_attn_workspace_bytes(cache, hq, n, most, width)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=dev) if size else None
    dargs = (cache, qd, _ints(start, dev), _ints(lens, dev), _ints(table_dev, dev), out, ws)
    sl = None if slopes is None else torch.from_numpy(slopes).to(dev)
    call = lambda s=stream: mbd.mbd_kv_attn(*dargs, max_new=most, scale=sc, softcap=softcap, window=window, slopes=sl, lse=lse, stream=s)
    kd, vd = kv.decode(c.k, fmt), kv.decode(c.v, fmt)
    args = [q, start, lens, table, kd, vd, c.ks, c.vs, bs, sc, softcap, window, slopes]
    ref, ref_lse, mine = kv.attention(*args)
    weight, _, _ = _abs_attention(args, np.abs(vd))
    for i in range(n):
        mine[start[i] + most:start[i + 1]] = False
    du = _tolerances(q, c, table, lens, start, bs, group, sc, softcap, slopes, ref, lens.max())
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 * 1.01 + 2 * du + (int(lens.max()) / 16 + 64) * 2.0 ** -24) * weight + 1e-30

    def check(tag=""):
        o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
        assert (o[~mine] == 7).all() and (l[~mine] == 7).all(), tag
        if qpad:
            assert (out_wide[:, hq * dim:] == 7).all(), tag
        assert np.isfinite(o).all(), tag
        off = np.abs(o - ref)[mine] - tol[mine]
        assert (off <= 0).all(), "%s worst %.3g over its tolerance, at %s" % (tag, off.max(), np.unravel_index(off.argmax(), off.shape))
        empty = np.isneginf(ref_lse) & mine[:, None]
        assert np.isneginf(l[empty]).all() and (o[empty] == 0).all(), tag
        some = mine[:, None] & ~empty
        np.testing.assert_allclose(l[some], ref_lse[some], atol=du + 2.0 ** -19, rtol=2.0 ** -21, err_msg=tag)
    return call, check, (out_wide, lse, ws)


def _run_attn(dev, *a, **kw):
    print("case attn", a, kw, flush=True)
    call, check, _ = _attn_case(dev, *a, **kw)
    call()
    torch.cuda.synchronize()
    check()


LENGTHS = [[1], [15], [16], [17], [33], [127], [128], [129], [640], [2, 1000, 64, 31, 1, 513]]


@pytest.mark.parametrize("fmt", [INT8, E4M3])
@pytest.mark.parametrize("lens", LENGTHS)
def test_attn_lengths(dev, fmt, lens):
    _run_attn(dev, fmt, 128, 16, 2, 4, lens, [1] * len(lens))


@pytest.mark.parametrize("fmt", [INT8, E4M3])
@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("hkv,group", [(1, 1), (3, 1), (1, 8), (2, 16), (1, 17), (1, 40), (1, 71)])
def test_attn_heads_and_dims(dev, fmt, dim, hkv, group):
    _run_attn(dev, fmt, dim, 32, hkv, group, [70, 200], [1, 1], pad=1)


@pytest.mark.parametrize("bs", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("fmt", [INT8, E4M3])
def test_attn_block_sizes(dev, fmt, bs):
    _run_attn(dev, fmt, 64, bs, 2, 3, [bs - 1, bs, bs + 1, 3 * bs + 5], [1, 1, 1, 1])


@pytest.mark.parametrize("fmt", [INT8, E4M3])
@pytest.mark.parametrize("new", [[5, 5, 5], [1, 16, 7], [0, 3, 0], [2, 0, 9]])
@pytest.mark.parametrize("dim,group", [(128, 4), (64, 1), (256, 3), (192, 8)])
def test_attn_verify(dev, fmt, new, dim, group):
    _run_attn(dev, fmt, dim, 16, 2, group, [max(37, new[0]), 300, 1100], new, pad=2, qpad=16)


@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("fmt", [INT8, E4M3])
def test_attn_prompts(dev, fmt, dim):
    _run_attn(dev, fmt, dim, 64, 1, 3, [150, 90], [150, 41], pad=1)


@pytest.mark.parametrize("fmt", [INT8, E4M3])
@pytest.mark.parametrize("opts", [dict(softcap=5.0), dict(window=1), dict(window=16), dict(window=100), dict(window=5000), dict(alibi=True),
                                  dict(softcap=20.0, window=70, alibi=True), dict(scale=0.0), dict(scale=-0.3), dict(softcap=0.5, scale=3.0)])
@pytest.mark.parametrize("dim,new", [(128, [1, 1, 1]), (64, [5, 3, 16]), (256, [40, 2, 9])])
def test_attn_masks_and_biases(dev, fmt, opts, dim, new):
    _run_attn(dev, fmt, dim, 16, 2, 2, [40, 333, 1500], new, **opts)


@pytest.mark.parametrize("fmt", [INT8, E4M3])
def test_attn_empty_rows(dev, fmt):
    """Requests with nothing cached, or less than they bring: rows that see no token; a
    request past max_new; requests whose blocks are all left out, or some."""
    _run_attn(dev, fmt, 128, 16, 1, 2, [0, 3, 50], [1, 5, 2])
    _run_attn(dev, fmt, 64, 16, 1, 2, [0], [3], window=4)
    _run_attn(dev, fmt, 128, 16, 2, 2, [40, 30, 64], [4, 2, 7], max_new=3)
    _run_attn(dev, fmt, 128, 16, 1, 2, [64, 700, 20], [1, 2, 1], holes=[(0, 1), (1, 0), (1, 7), (1, 43), (2, 0), (2, 1)])


@pytest.mark.parametrize("fmt", [INT8, E4M3])
def test_attn_split_long(dev, fmt):
    """Long requests beside short ones: parts joined from the workspace."""
    _run_attn(dev, fmt, 128, 64, 1, 8, [20000, 1, 300, 4097], [1, 1, 1, 1])
    _run_attn(dev, fmt, 64, 16, 2, 2, [6001, 50], [5, 2], softcap=30.0, window=4000)


@pytest.mark.parametrize("fmt", [INT8, E4M3])
def test_attn_prompts_beside_decodes(dev, fmt):
    """One call with prompt slices, verify steps and single tokens of long contexts: row tiles
    and parts of requests in one row of work, some of it joined."""
    _run_attn(dev, fmt, 128, 64, 2, 4, [260, 9000, 33, 5000, 64], [130, 1, 5, 1, 64], pad=2)
    _run_attn(dev, fmt, 64, 16, 1, 40, [50, 3000, 3000], [9, 4, 1], window=2500)


def test_attn_row_tiles_beyond_places(dev):
    """More tiles of query rows than the chip has places for a head's workgroups, next to a
    request that is still cut."""
    _run_attn(dev, E4M3, 256, 32, 4, 16, [9000] + [24] * 70, [1] + [24] * 70)


def test_attn_wide_cap_is_no_cap(dev):
    """A cap far above every score leaves them as they are: cap tanh(u / cap) = u - u^3 / (3 cap^2) + ..,
    so with |u| < 100 and a cap of 1e6 within 1e-6, far inside the tolerance of the uncapped call."""
    call, check, (out, lse, _) = _attn_case(dev, INT8, 128, 16, 2, 2, [300, 90], [2, 1])
    call()
    torch.cuda.synchronize()
    check()
    want, wlse = out.float().clone(), lse.clone()
    capped, _, (out, lse, _) = _attn_case(dev, INT8, 128, 16, 2, 2, [300, 90], [2, 1], softcap=1e6)
    capped()
    torch.cuda.synchronize()
    assert (lse - wlse).abs().max().item() <= 2.0 ** -16
    # scores that close move a bf16 weight or output by one of its steps at most
    assert ((out.float() - want).abs() <= 2.0 ** -7 * want.abs() + 2.0 ** -9 * want.abs().max()).all()


def test_attn_many_requests(dev):
    _run_attn(dev, INT8, 64, 16, 1, 2, list(np.random.default_rng(1).integers(1, 60, 300)), [1] * 300)


@pytest.mark.parametrize("fmt", [INT8, E4M3])
@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("hkv,group,new,opts", [
    (16, 2, 1, {}), (16, 5, 3, {}), (16, 1, 1, dict(softcap=9.0, window=200, alibi=True))])
def test_attn_more_requests_than_places(dev, fmt, dim, hkv, group, new, opts):
    """So many requests that one wave works on each part; a long one among them is cut, some see nothing."""
    n = 70
    lens = list(np.random.default_rng(2).integers(new, 100, n))
    lens[1] = 1500
    _run_attn(dev, fmt, dim, 16, hkv, group, lens, [i % (new + 1) if i else 0 for i in range(n - 1)] + [new], **opts)


def test_attn_most_requests(dev):
    """4096 requests, the most, of which three in four are not in the step."""
    n = 4096
    lens = list(np.random.default_rng(3).integers(1, 5, n))
    lens[-1], lens[2000] = 700, 100
    _run_attn(dev, E4M3, 64, 16, 1, 1, lens, [int(i % 4 == 3) for i in range(n)])


def test_attn_more_heads_than_places(dev):
    _run_attn(dev, INT8, 64, 16, 1100, 1, [20, 40, 3], [1, 0, 1])


def test_attn_large_scores(dev):
    """Scores far apart: running maxima that move late, weights that underflow."""
    _run_attn(dev, INT8, 128, 16, 1, 4, [900], [3], scale=8.0)


def test_attn_offsets_past_32_bits(dev):
    """Blocks whose byte offsets pass 2^32: a cache of 5 GB, of which a few blocks are used."""
    mbd = _mbd()
    hkv, dim, bs = 8, 256, 256
    blocks = 5 * (1 << 30) // (hkv * dim * bs)
    assert (blocks - 1) * hkv * dim * bs > 1 << 32
    codes = [torch.empty((blocks, hkv, bs * dim), dtype=torch.uint8, device=dev) for _ in range(2)]
    scales = [torch.empty((blocks, hkv), device=dev) for _ in range(2)]
    cache = mbd.KvCache(mbd.MBD_KV_INT8, bs, dim, *codes, *scales)
    rng = np.random.default_rng(4)
    table = np.array([[blocks - 1, 0], [blocks - 2, blocks - 3]])
    lens = np.array([300, 400])
    slots = np.concatenate([[table[i][p // bs] * bs + p % bs for p in range(lens[i])] for i in range(2)])
    x = torch.from_numpy(rng.standard_normal((700, hkv, 2, dim))).to(torch.bfloat16)
    mbd.mbd_kv_append(cache, x[:, :, 0].contiguous().to(dev), x[:, :, 1].contiguous().to(dev), _ints(slots, dev))
    ko, vo = torch.empty((700, hkv, dim), device=dev), torch.empty((700, hkv, dim), device=dev)
    mbd.mbd_kv_gather(cache, _ints(slots, dev), ko, vo)
    q = torch.from_numpy(rng.standard_normal((2, hkv, dim))).to(torch.bfloat16).to(dev)
    out = torch.zeros_like(q)
    ws = torch.empty(mbd.mbd_kv_attn_workspace_bytes(cache, hkv, 2, 1, 2), dtype=torch.uint8, device=dev)
    mbd.mbd_kv_attn(cache, q, _ints([0, 1, 2], dev), _ints(lens, dev), _ints(table, dev), out, ws)
    torch.cuda.synchronize()
    amax = x.float().abs().amax().item()
    for o, j in ((ko, 0), (vo, 1)):
        assert (o.cpu() - x[:, :, j].float()).abs().max().item() <= 0.5001 * amax / 127
    k, v, qf = ko.double().cpu(), vo.double().cpu(), q.double().cpu()
    for i, (a, b) in enumerate(((0, 300), (300, 700))):
        w = torch.softmax(torch.einsum("hd,thd->ht", qf[i], k[a:b]) * dim ** -0.5, 1)
        ref, mag = torch.einsum("ht,thd->hd", w, v[a:b]), torch.einsum("ht,thd->hd", w, v[a:b].abs())
        assert ((out[i].double().cpu() - ref).abs() <= 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -13) * mag).all()


# ------------------------------------------------------------------ streams, graphs, a step

def test_attn_other_stream_and_graph(dev):
    call, check, (out, lse, ws) = _attn_case(dev, E4M3, 128, 16, 2, 4, [700, 3, 90], [2, 1, 5])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(side.cuda_stream)
    side.synchronize()
    check("side stream")
    want = out.clone(), lse.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(None)
    for i in range(3):
        out.fill_(7.0)
        lse.fill_(7.0)
        if ws is not None:
            ws.fill_(0xFF)                            # eager work between replays
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]), "replay %d" % i


def test_attn_repeats_bit_for_bit(dev):
    call, check, (out, lse, ws) = _attn_case(dev, INT8, 128, 32, 4, 4, [5000, 700, 9], [1, 1, 1])
    got = []
    for _ in range(3):
        call()
        torch.cuda.synchronize()
        got.append((out.clone(), lse.clone()))
    assert all(torch.equal(a, got[0][0]) and torch.equal(b, got[0][1]) for a, b in got)


@pytest.mark.parametrize("fmt", [INT8, E4M3])
@pytest.mark.parametrize("graph", [False, True])
def test_decode_steps(dev, fmt, graph):
    """A run as it is used: prompts, then verify steps of 4 tokens of which some are taken
    back, then an ended request whose blocks another takes; slots -> append -> attention ->
    an INT4 output projection, every step against the oracle on the same inputs."""
    import synth
    from oracle import gemv, int4
    mbd = _mbd()
    rng = np.random.default_rng(11)
    n, hkv, group, dim, bs, width, blocks = 3, 2, 2, 64, 16, 6, 14
    hq, T = hkv * group, 60
    c = Cache(fmt, blocks, hkv, dim, bs, dev)
    cache = c.device()
    pool = mbd.KvPool(bs, torch.full((n, width), -1, dtype=torch.int32, device=dev), _ints(np.arange(blocks), dev))
    table, free = np.full((n, width), -1), np.arange(blocks)
    z = lambda s: torch.zeros(s, dtype=torch.int32, device=dev)
    lens, held, n_free, new_dev = z(n), z(n), _ints([blocks], dev), z(n)
    start, slots, pos, status = z(n + 1), z(T), z(T), z(n)
    w = synth.f32_to_bf16_bits((rng.standard_t(4, (128, hq * dim)) * 0.02).astype(np.float32))
    proj = mbd.to_device(mbd.mbd_pack(mbd.MBD_INT4_G128, w), dev)
    qw, sw = int4.quantize(w)
    qkv = torch.zeros((T, (hq + 2 * hkv) * dim), dtype=torch.bfloat16, device=dev)
    q, k, v = (qkv[:, a * dim:b * dim].unflatten(1, (b - a, dim)) for a, b in ((0, hq), (hq, hq + hkv), (hq + hkv, hq + 2 * hkv)))
    out = torch.zeros((T, hq, dim), dtype=torch.bfloat16, device=dev)
    y = torch.zeros((16, 128), device=dev)
    ws = torch.empty(mbd.mbd_kv_attn_workspace_bytes(cache, hq, n, 50, width), dtype=torch.uint8, device=dev)

    def step():
        mbd.mbd_kv_slots(pool, new_dev, lens, held, n_free, start, slots, pos, lens, held, n_free, status)
        mbd.mbd_kv_append(cache, k, v, slots)
        mbd.mbd_kv_attn(cache, q, start, lens, pool.block_table, out, ws, max_new=50)
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
        for t, name in ((start, "seq_start"), (slots, "slots"), (pos, "positions"), (lens, "lens_out"), (held, "held_out"), (n_free, "n_free_out"),
                        (status, "status")):
            np.testing.assert_array_equal(t.cpu().numpy(), np.atleast_1d(ref[name]), err_msg="%s of step %d" % (name, s))
        r_lens, r_held, r_free = ref["lens_out"], ref["held_out"], ref["n_free_out"]
        xn = x.double().numpy().reshape(T, -1, dim)
        kv.append(c.k, c.ks, xn[:, hq:hq + hkv], ref["slots"], fmt)
        kv.append(c.v, c.vs, xn[:, hq + hkv:], ref["slots"], fmt)
        kd, vd = kv.decode(c.k, fmt), kv.decode(c.v, fmt)
        args = [xn[:, :hq], ref["seq_start"], r_lens, table, kd, vd, c.ks, c.vs, bs, dim ** -0.5]
        want, lse, mine = kv.attention(*args)
        mag, _, _ = _abs_attention(args, np.abs(vd))
        du = 2.0 ** -23 * (dim + 8) * dim ** -0.5 * np.abs(xn).max() ** 2 * dim
        o = out.double().cpu().numpy()
        tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -8 * 1.01 + 2 * du + 2.0 ** -17) * mag + 1e-30
        assert (np.abs(o - want) <= tol)[mine].all(), "step %d" % s
        obits = out[:16].flatten(1).cpu().view(torch.int16).numpy().view(np.uint16)
        assert gemv.rel_l2(y.cpu().numpy().astype(np.float64), gemv.gemv(int4.dequant(qw, sw), obits)) <= 1e-3
        lens -= _ints(back, dev)                        # drafts that were not accepted
        r_lens = r_lens - np.array(back)


def test_two_streams_with_their_own_workspaces(dev):
    """Two calls in flight at once, each with its own workspace and outputs."""
    a = _attn_case(dev, INT8, 128, 16, 1, 4, [3000, 70], [1, 1], seed=1)
    b = _attn_case(dev, E4M3, 64, 16, 2, 2, [2500, 9], [3, 2], seed=2)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        for (call, _, _), s in zip((a, b), streams):
            call(s.cuda_stream)
    torch.cuda.synchronize()
    a[1]("first")
    b[1]("second")


def test_nothing_to_do(dev):
    """No rows, no new tokens: nothing written, nothing launched out of range."""
    mbd = _mbd()
    c = Cache(INT8, 4, 1, 64, 16, dev)
    cache = c.device()
    empty = torch.empty((0, 1, 64), dtype=torch.bfloat16, device=dev)
    none = torch.empty(0, dtype=torch.int32, device=dev)
    mbd.mbd_kv_append(cache, empty, empty, none)
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
    c = Cache(INT8, 8, 1, 64, 16, dev)
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


@pytest.mark.parametrize("fmt", [INT8, E4M3])
@pytest.mark.parametrize("scale,softcap,key_scale", [(2.0 ** 64, 0.0, 2.0 ** 100), (2.0 ** 64, 2.0 ** -62, 2.0 ** 20), (-2.0 ** 64, 1.0, 2.0 ** 100),
                                                     (2.0 ** 10, 2.0, 2.0 ** 120)])
def test_attn_factors_past_fp32(dev, fmt, scale, softcap, key_scale):
    """The factor of a block's scores (key scale x scale / cap) passes fp32: a zero score is 0 all the
    same, any other meets the cap.  One query channel at most is not zero, so that every product
    is exact and no rounding decides a score's sign; without a cap the queries are zero."""
    mbd = _mbd()
    print("case far factors", fmt, scale, softcap, key_scale, flush=True)
    dim, bs, length, n = 64, 16, 40, 2
    c = Cache(fmt, 4, 1, dim, bs, dev)
    c.fill(np.arange(4))
    c.ks[:] = key_scale
    c.k[1], c.ks[1] = 0, 0                              # a block of zero tokens
    table, start, lens = np.array([[2, 1, 0], [3, -1, -1]]), np.array([0, 1, 2]), np.array([length, 9])
    q = np.zeros((n, 2, dim))
    if softcap:
        q[:, 0, 5] = 1.0
    cache = c.device()
    out = torch.full((n, 2, dim), 7.0, dtype=torch.bfloat16, device=dev)
    lse = torch.full((n, 2), 7.0, device=dev)
    ws = torch.empty(max(16, mbd.mbd_kv_attn_workspace_bytes(cache, 2, n, 1, 3)), dtype=torch.uint8, device=dev)
    mbd.mbd_kv_attn(cache, torch.from_numpy(q).to(torch.bfloat16).to(dev), _ints(start, dev), _ints(lens, dev), _ints(table, dev), out, ws, scale=scale,
                    softcap=softcap, lse=lse)
    torch.cuda.synchronize()
    args = [q, start, lens, table, kv.decode(c.k, fmt), kv.decode(c.v, fmt), c.ks, c.vs, bs, scale, softcap]
    ref, ref_lse, _ = kv.attention(*args)
    weight, _, _ = _abs_attention(args, np.abs(kv.decode(c.v, fmt)))
    # scores are 0 or +-cap, up to the cap's own rounding: the bounds of _tolerances without their products
    du = 2.0 ** -20 * softcap
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 * 1.01 + 2 * du + 2.0 ** -17) * weight
    assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()
    np.testing.assert_allclose(lse.double().cpu().numpy(), ref_lse, atol=du + 2.0 ** -19, rtol=2.0 ** -21)


@pytest.mark.parametrize("fmt", [INT8, E4M3])
@pytest.mark.parametrize("heads", [2, 700])
def test_append_ties_over_any_stored_scale(dev, fmt, heads):
    """Blocks whose stored scale is no power of two (a cache filled by another program), appended to
    with values in the middle between two codes: the code comes from the fp32 quotient, to even.
    With many heads the call is large enough for the kernel over windows of tokens."""
    mbd = _mbd()
    print("case stored scales", fmt, heads, flush=True)
    blocks, dim, bs = 12, 64, 16
    c = Cache(fmt, blocks, heads, dim, bs, dev, seed=heads)
    c.fill(np.arange(blocks))
    c.ks[:] = np.float32(np.exp2(c.rng.uniform(-9, 3, c.ks.shape)))
    c.vs[:] = np.float32(np.exp2(c.rng.uniform(-9, 3, c.vs.shape)))
    fill = c.rng.integers(1, bs - 1, blocks)
    live = fill + c.rng.integers(1, bs - fill + 1)
    _live_only(c, fill)
    slots = np.concatenate([b * bs + np.arange(fill[b], live[b]) for b in range(blocks)])
    block = slots // bs
    values = kv.decode(np.arange(127), fmt) if fmt == E4M3 else np.arange(128.0)
    mids = (values[1:] + values[:-1]) / 2
    pick = lambda: c.rng.choice(mids, (len(slots), heads, dim)) * c.rng.choice([-1, 1], (len(slots), heads, dim))
    k, v = (np.float32(pick() * s[block][..., None].astype(np.float64)) for s in (c.ks, c.vs))
    v[::3] *= np.float32(1.7)                           # some blocks' scales grow, by what is no power of two
    cache = c.device()
    mbd.mbd_kv_append(cache, torch.from_numpy(k).to(dev), torch.from_numpy(v).to(dev), _ints(slots, dev))
    torch.cuda.synchronize()
    kv.append(c.k, c.ks, k, slots, fmt)
    kv.append(c.v, c.vs, v, slots, fmt)
    got = {n: t.cpu().numpy() for n, t in cache.tensors.items()}
    np.testing.assert_array_equal(got["k_scale"], c.ks)
    np.testing.assert_array_equal(got["v_scale"], c.vs)
    gk, gv = kv.unpack(got["k_codes"], bs, dim, False), kv.unpack(got["v_codes"], bs, dim, True)
    for b in range(blocks):
        np.testing.assert_array_equal(gk[b, :, :live[b]], c.k[b, :, :live[b]], err_msg="keys of block %d" % b)
        np.testing.assert_array_equal(gv[b, :, :live[b]], c.v[b, :, :live[b]], err_msg="values of block %d" % b)


WINDOW_APPENDS = [  # heads, dim, bs, (cached, new) of each request; all large enough for the kernel over windows of tokens
    (40, 64, 16, [(0, 70), (5, 40), (16, 33), (31, 1), (0, 16), (15, 50)]),
    (24, 128, 16, [(3, 200), (0, 97), (15, 1), (9, 7), (32, 64)]),
    (17, 192, 32, [(30, 150), (7, 3), (0, 260), (31, 2), (17, 88)]),
    (16, 256, 64, [(63, 300), (1, 62), (0, 129), (20, 44)]),
    (12, 128, 128, [(0, 400), (100, 250), (127, 2), (64, 64)]),
    (10, 64, 256, [(0, 600), (200, 300), (16, 128), (255, 1), (17, 239)]),
    (9, 256, 256, [(3, 900), (40, 216), (128, 1)]),
    (9, 192, 64, [(13, 1000), (0, 5), (60, 4)]),
    (66, 64, 256, [(3, 700), (250, 300), (0, 40), (16, 1)]),       # windows of 64 tokens, the widest
    (70, 128, 16, [(7, 900), (0, 33), (31, 1), (5, 60)]),
]


@pytest.mark.parametrize("fmt", [INT8, E4M3])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("special", [False, True])
@pytest.mark.parametrize("heads,dim,bs,requests", WINDOW_APPENDS)
def test_append_prompts(dev, fmt, dtype, special, heads, dim, bs, requests):
    """Prompts: runs that a whole workgroup takes, over windows of tokens, beside short ones; they begin and
    end inside tiles, over codes of before whose scale grows or stays, go past a window and past 128 tokens of
    a block, with rows of no slot between requests and, if special, infinities and NaN."""
    mbd = _mbd()
    print("case prompts", fmt, dtype, special, heads, dim, bs, requests, flush=True)
    ends = np.array([a + b for a, b in requests])
    held = -(-ends // bs)
    blocks = int(held.sum()) + 2
    c = Cache(fmt, blocks, heads, dim, bs, dev, seed=heads + bs)
    order, at = c.rng.permutation(blocks), 0
    slots, before, live = [], np.zeros(blocks, int), np.zeros(blocks, int)
    for i, (cached, new) in enumerate(requests):
        table = order[at:at + held[i]]
        at += held[i]
        place = np.arange(cached + new)
        to = table[place // bs] * bs + place % bs
        for s, p in zip(to, place):
            live[s // bs] = s % bs + 1
            if p < cached:
                before[s // bs] = s % bs + 1
        slots += list(to[cached:]) + ([-1] if i % 2 else [])
    slots = np.array(slots + [blocks * bs, -2 ** 31])
    T, row = len(slots), heads * dim
    assert T * 2 * heads > 16384
    c.fill(np.flatnonzero(before))
    c.ks[::2] *= np.float32(0.25)                       # every other block's keys, and the others' values, outgrow their scale
    c.vs[1::2] *= np.float32(0.25)
    _live_only(c, before)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x = torch.from_numpy(c.rng.standard_normal((T, 2 * row + 8)) * c.rng.choice([0.3, 1.0], (T, 1))).to(dt)
    if special:
        for value in (float("inf"), float("-inf"), float("nan")):
            x[torch.from_numpy(c.rng.integers(0, T, 40)), torch.from_numpy(c.rng.integers(0, 2 * row, 40))] = value
        x[2:5, :dim] = float("inf")
    cache, d = c.device(), x.to(dev)
    mbd.mbd_kv_append(cache, d[:, :row].unflatten(1, (heads, dim)), d[:, row:2 * row].unflatten(1, (heads, dim)), _ints(slots, dev))
    torch.cuda.synchronize()
    xn = x.double().numpy()
    kv.append(c.k, c.ks, xn[:, :row].reshape(T, heads, dim), slots, fmt)
    kv.append(c.v, c.vs, xn[:, row:2 * row].reshape(T, heads, dim), slots, fmt)
    got = {n: t.cpu().numpy() for n, t in cache.tensors.items()}
    used = live > 0
    np.testing.assert_array_equal(got["k_scale"][used], c.ks[used])
    np.testing.assert_array_equal(got["v_scale"][used], c.vs[used])
    assert np.isnan(got["k_scale"][~used]).all() and np.isnan(got["v_scale"][~used]).all()
    gk, gv = kv.unpack(got["k_codes"], bs, dim, False), kv.unpack(got["v_codes"], bs, dim, True)
    for b in range(blocks):
        np.testing.assert_array_equal(gk[b, :, :live[b]], c.k[b, :, :live[b]], err_msg="keys of block %d" % b)
        np.testing.assert_array_equal(gv[b, :, :live[b]], c.v[b, :, :live[b]], err_msg="values of block %d" % b)


EVERY = [  # head_dim, KV heads, query heads a KV head, tokens, short requests beside, new tokens, window
    (64, 8, 16, 20000, 0, 1, 0),         # parts of four waves
    (128, 4, 8, 4097, 3, 1, 0),
    (64, 16, 4, 4097, 69, 1, 0),         # more requests than places: parts of one wave
    (128, 2, 16, 4100, 2, 5, 0),         # two row tiles
    (256, 1, 16, 1500, 1, 3, 0),
    (64, 4, 16, 6000, 2, 1, 2500),       # a window that begins inside a tile
    (192, 1, 16, 3000, 1, 4, 1001),
]


@pytest.mark.parametrize("fmt", [INT8, E4M3])
@pytest.mark.parametrize("dim,hkv,group,length,others,new,window", EVERY)
def test_attn_every_position(dev, fmt, dim, hkv, group, length, others, new, window):
    """Every cached position counts once.  Keys and values hold their position's 15 bits as +-1.5, a query
    the bits of the position that it looks for: its score is 24 * 15, any other's at least 48 lower, so
    o is that position's value (the weight and the output each rounded by at most 2^-8) and lse its
    score (a few fp32 roundings of 360 * log2(e)); a lost token moves lse by 48, one taken twice by log 2.
    Queries of zero weigh all tokens alike: sums of ones are exact, lse is log(count) up to the
    logarithm's and the product's roundings."""
    mbd = _mbd()
    print("case every position", fmt, dim, hkv, group, length, others, new, window, flush=True)
    bs, hq, n = 32, hkv * group, others + 1
    mid = others // 2
    lens, fresh = np.full(n, 3), np.ones(n, int)
    lens[mid], fresh[mid] = length, new
    held = -(-lens // bs)
    c = Cache(fmt, int(held.sum()), hkv, dim, bs, dev)
    order = c.rng.permutation(int(held.sum()))
    table, at = np.full((n, held.max()), -1), 0
    for i in range(n):
        table[i, :held[i]] = order[at:at + held[i]]
        at += held[i]
    c.ks[:] = c.vs[:] = 2.0 ** -6
    bits = lambda p: ((np.asarray(p)[..., None] >> np.arange(15)) & 1) * 2 - 1
    for i in range(n):
        place = np.arange(held[i] * bs)
        live = place < lens[i]
        plus, minus = (int(kv.encode(np.array([96.0 * s]), fmt)[0]) for s in (1, -1))
        codes = np.zeros((len(place), dim), np.uint8)
        codes[:, :15] = np.where(bits(place) > 0, plus, minus)
        for store in (c.k, c.v):
            store[table[i, place[live] // bs], :, place[live] % bs] = codes[live][:, None]
    cache = c.device()
    start = np.concatenate([[0], np.cumsum(fresh)])
    T, row0 = int(start[-1]), int(start[mid])
    size = mbd.mbd_kv_attn_workspace_bytes(cache, hq, n, new, table.shape[1])
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=dev) if size else None
    q = torch.zeros((T, hq, dim), dtype=torch.bfloat16, device=dev)
    out, lse = torch.zeros_like(q), torch.zeros((T, hq), device=dev)
    ints = _ints(start, dev), _ints(lens, dev), _ints(table, dev)
    call = lambda: mbd.mbd_kv_attn(cache, q, *ints, out, ws, max_new=new, scale=16.0, window=window, lse=lse)
    call()
    torch.cuda.synchronize()
    pos = np.repeat(lens, fresh) - np.repeat(start[1:], fresh) + np.arange(T)
    count = np.minimum(pos + 1, window) if window else pos + 1
    np.testing.assert_allclose(lse.double().cpu().numpy(), np.repeat(np.log(count)[:, None], hq, 1), rtol=2.0 ** -21, atol=2.0 ** -24)
    seen = np.arange(max(0, length - window) if window else 0, length - new + 1)     # by every row of the request
    per = new * hq
    tol_lse = 360 * 2.0 ** -21
    for a in range(0, len(seen), per):
        target = np.resize(seen[a:a + per], per).reshape(new, hq)
        q[row0:row0 + new, :, :15] = torch.from_numpy(bits(target)).to(torch.bfloat16).to(dev)
        call()
        torch.cuda.synchronize()
        o, l = out[row0:row0 + new].double().cpu().numpy(), lse[row0:row0 + new].double().cpu().numpy()
        off = np.abs(o[..., :15] - 1.5 * bits(target))
        assert off.max() <= 1.5 * (2.0 ** -7 + 2.0 ** -14), "position %d" % target.ravel()[off.max(-1).argmax()]
        assert (o[..., 15:] == 0).all()
        gap = np.abs(l - 360)
        assert gap.max() <= tol_lse, "position %d" % target.ravel()[gap.argmax()]


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("dim,hkv,group,lens,new", [(128, 2, 4, [700, 40], [2, 1]), (64, 1, 8, [90, 2000, 33], [5, 9, 1]), (256, 2, 1, [50] * 3, [1] * 3)])
def test_attn_bad_queries_stay_in_their_row(dev, dim, hkv, group, lens, new, bad):
    """A query of NaN or infinities leaves every other row's output and lse as they are, bit for bit."""
    mbd = _mbd()
    print("case bad queries", dim, hkv, group, lens, new, bad, flush=True)
    bs, hq, n = 16, hkv * group, len(lens)
    held = -(-np.array(lens) // bs)
    c = Cache(INT8, int(held.sum()), hkv, dim, bs, dev)
    c.fill(np.arange(int(held.sum())))
    table = np.full((n, held.max()), -1)
    for i in range(n):
        table[i, :held[i]] = held[:i].sum() + np.arange(held[i])
    cache, start = c.device(), np.concatenate([[0], np.cumsum(new)])
    T = int(start[-1])
    q = torch.from_numpy(c.rng.standard_normal((T, hq, dim))).to(torch.bfloat16).to(dev)
    out, lse = torch.zeros_like(q), torch.zeros((T, hq), device=dev)
    ws = torch.empty(max(16, mbd.mbd_kv_attn_workspace_bytes(cache, hq, n, max(new), table.shape[1])), dtype=torch.uint8, device=dev)
    call = lambda: mbd.mbd_kv_attn(cache, q, _ints(start, dev), _ints(lens, dev), _ints(table, dev), out, ws, max_new=max(new), lse=lse)
    call()
    want, want_lse = out.clone(), lse.clone()
    keep = torch.ones((T, hq), dtype=torch.bool, device=dev)
    for row, head, channel in ((0, 0, 0), (T - 1, hq - 1, dim - 1), (T // 2, hq // 2, slice(None))):
        q[row, head, channel] = bad
        keep[row, head] = False
    call()
    torch.cuda.synchronize()
    assert torch.equal(out[keep], want[keep]) and torch.equal(lse[keep], want_lse[keep])
    assert not torch.isfinite(out[~keep].float()).all(-1).any()


@pytest.mark.parametrize("seed,n,bs,width,prompt_hi", [(10, 700, 16, 40, 300), (11, 90, 64, 30, 1500), (12, 1500, 32, 12, 90)])
@pytest.mark.parametrize("in_place", [False, True])
def test_slots_of_many_tokens(dev, seed, n, bs, width, prompt_hi, in_place):
    """Steps whose slot map one workgroup writes, or the whole chip, just below and above where that changes."""
    mbd = _mbd()
    new, lens, held, table, free, n_free = _requests(seed, n, bs, width, prompt_hi)
    total = int(np.maximum(new, 0).sum())
    assert total > 8192
    for T in (8192, 8193, total + 5):
        print("case slots of many tokens", seed, n, bs, width, in_place, T, flush=True)
        ref_table, ref_free = table.copy(), free.copy()
        ref = kv.slots(new, lens, held, ref_table, ref_free, n_free, bs, T)
        pool = mbd.KvPool(bs, _ints(table, dev), _ints(free, dev))
        d = {k: _ints(v, dev) for k, v in dict(new=new, lens=lens, held=held, n_free=[n_free]).items()}
        o = {k: torch.full((s,), -55, dtype=torch.int32, device=dev) for k, s in dict(
            seq_start=n + 1, slots=T, positions=T, lens_out=n, held_out=n, n_free_out=1, status=n).items()}
        if in_place:
            o["lens_out"], o["held_out"], o["n_free_out"] = d["lens"], d["held"], d["n_free"]
        mbd.mbd_kv_slots(pool, d["new"], d["lens"], d["held"], d["n_free"], o["seq_start"], o["slots"], o["positions"], o["lens_out"],
                         o["held_out"], o["n_free_out"], o["status"])
        torch.cuda.synchronize()
        for name, want in ref.items():
            np.testing.assert_array_equal(o[name].cpu().numpy(), np.atleast_1d(want), err_msg="%s, T %d" % (name, T))
        np.testing.assert_array_equal(pool.block_table.cpu().numpy(), ref_table)
        np.testing.assert_array_equal(pool.free_blocks.cpu().numpy(), ref_free)
