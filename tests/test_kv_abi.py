"""Argument checks of the KV-cache calls: each refusal with its status, before any GPU
work (fake pointers, never dereferenced), and the binding's own checks."""
import ctypes

import pytest

mbd = pytest.importorskip("memory_bound_decode_amd")
torch = pytest.importorskip("torch")

P = 0x10000


@pytest.fixture(scope="module")
def L():
    try:
        return mbd.lib()
    except ImportError as e:                         # pragma: no cover
        pytest.skip(str(e))


def _cache(**kw):
    d = dict(fmt=mbd.MBD_KV_INT8, block_size=16, n_heads=2, head_dim=128, n_blocks=8, k_codes=P, v_codes=P, k_scale=P, v_scale=P)
    return mbd.MbdKvCache(**(d | kw))


BAD_CACHES = [(dict(fmt=9), "EINVAL"), (dict(block_size=24), "ESHAPE"), (dict(block_size=512), "ESHAPE"), (dict(head_dim=96), "ESHAPE"),
              (dict(head_dim=320), "ESHAPE"), (dict(n_heads=0), "ESHAPE"), (dict(n_blocks=0), "ESHAPE"), (dict(n_blocks=1 << 27), "ESHAPE"),
              (dict(k_codes=None), "EINVAL"), (dict(v_scale=None), "EINVAL"), (dict(v_codes=P + 8), "EALIGN"), (dict(k_scale=P + 2), "EALIGN")]


@pytest.mark.parametrize("change,status", BAD_CACHES)
def test_bad_caches(L, change, status):
    want = getattr(mbd, "MBD_" + status)
    c = _cache(**change)
    assert L.mbd_kv_append(ctypes.byref(c), P, P, mbd.MBD_BF16, 256, 256, P, 1, None) == want
    assert L.mbd_kv_gather(ctypes.byref(c), P, 1, mbd.MBD_F32, P, P, None) == want
    assert L.mbd_kv_attn(ctypes.byref(c), ctypes.byref(_args()), P, P, P, P, P, None, P, 1 << 30, None) == want
    assert L.mbd_last_error()


def test_append_and_gather_arguments(L):
    c = ctypes.byref(_cache())
    app = lambda k=P, v=P, dt=mbd.MBD_BF16, ks=256, vs=256, s=P, T=1: L.mbd_kv_append(c, k, v, dt, ks, vs, s, T, None)
    assert L.mbd_kv_append(None, P, P, 1, 256, 256, P, 1, None) == mbd.MBD_EINVAL
    assert app(k=None) == app(s=None) == app(dt=3) == mbd.MBD_EINVAL
    assert app(k=P + 8) == app(v=P + 4) == app(s=P + 1) == mbd.MBD_EALIGN
    assert app(ks=255) == app(vs=248) == app(ks=260) == app(T=-1) == app(T=(1 << 24) + 1) == mbd.MBD_ESHAPE
    assert app(T=0, k=None, v=None, s=None) == mbd.MBD_OK
    gat = lambda s=P, T=1, dt=mbd.MBD_F32, k=P, v=P: L.mbd_kv_gather(c, s, T, dt, k, v, None)
    assert gat(k=None) == gat(s=None) == gat(dt=0) == mbd.MBD_EINVAL
    assert gat(k=P + 8) == mbd.MBD_EALIGN and gat(T=-1) == mbd.MBD_ESHAPE and gat(T=0) == mbd.MBD_OK


def test_slots_arguments(L):
    base = dict(n_seqs=4, block_size=16, max_blocks=8, n_blocks=100, block_table=P, free_blocks=P)

    def call(T=4, at=None, value=None, **kw):
        pool = mbd.MbdKvPool(**(base | kw))
        ptrs = [P] * 11
        if at is not None:
            ptrs[at] = value
        return L.mbd_kv_slots(ctypes.byref(pool), *ptrs[:4], T, *ptrs[4:], None)

    assert L.mbd_kv_slots(None, *[P] * 4, 1, *[P] * 7, None) == mbd.MBD_EINVAL
    for kw in (dict(n_seqs=0), dict(n_seqs=4097), dict(block_size=8), dict(max_blocks=0), dict(max_blocks=1 << 27), dict(n_blocks=0),
               dict(n_blocks=1 << 27), dict(T=-1)):
        assert call(**kw) == mbd.MBD_ESHAPE, kw
    assert call(block_table=None) == call(free_blocks=None) == mbd.MBD_EINVAL
    assert call(free_blocks=P + 2) == mbd.MBD_EALIGN
    for i in range(11):
        if i != 6:                                   # positions may be NULL
            assert call(at=i, value=None) == mbd.MBD_EINVAL, i
        assert call(at=i, value=P + 2) == mbd.MBD_EALIGN, i


def _args(**kw):
    d = dict(n_heads=8, n_seqs=2, max_blocks=4, T=2, max_new=1, window=0, scale=0.1, softcap=0.0, slopes=None, q_stride=1024, out_stride=1024)
    return mbd.MbdKvAttnArgs(**(d | kw))


BAD_ARGS = [(dict(n_heads=7), "ESHAPE"), (dict(n_heads=0), "ESHAPE"), (dict(n_seqs=0), "ESHAPE"), (dict(n_seqs=4097), "ESHAPE"),
            (dict(max_blocks=0), "ESHAPE"), (dict(max_blocks=(1 << 26) + 1), "ESHAPE"), (dict(max_blocks=1 << 26, n_seqs=32), "ESHAPE"),
            (dict(T=-1), "ESHAPE"), (dict(T=(1 << 24) + 1), "ESHAPE"), (dict(max_new=0), "ESHAPE"), (dict(max_new=1 << 22), "ESHAPE"),
            (dict(window=-1), "EINVAL"), (dict(scale=float("nan")), "EINVAL"), (dict(softcap=-1.0), "EINVAL"),
            (dict(softcap=float("inf")), "EINVAL"), (dict(softcap=float("nan")), "EINVAL"), (dict(n_heads=514), "ESHAPE"), (dict(softcap=1e-30), "EINVAL"), (dict(scale=float("inf")), "EINVAL"),
            (dict(scale=-1e30), "EINVAL"), (dict(n_seqs=4096, max_new=1 << 20, n_heads=8), "ESHAPE"), (dict(q_stride=1016), "ESHAPE"), (dict(out_stride=1028), "ESHAPE"),
            (dict(slopes=P + 2), "EALIGN"), (dict(n_heads=512, n_seqs=4096, max_new=1 << 15, T=1 << 24, q_stride=1 << 16, out_stride=1 << 16), "ESHAPE")]


@pytest.mark.parametrize("change,status", BAD_ARGS)
def test_bad_attention_arguments(L, change, status):
    c, a = _cache(), _args(**change)
    assert L.mbd_kv_attn(ctypes.byref(c), ctypes.byref(a), P, P, P, P, P, None, P, 1 << 40, None) == getattr(mbd, "MBD_" + status)


def test_attention_pointers_and_workspace(L):
    c = _cache()

    def call(a, **kw):
        d = dict(q=P, start=P, lens=P, table=P, out=P, lse=None, ws=P, size=1 << 40) | kw
        return L.mbd_kv_attn(ctypes.byref(c), None if a is None else ctypes.byref(a), d["q"], d["start"], d["lens"], d["table"], d["out"],
                             d["lse"], d["ws"], d["size"], None)

    a = _args(max_blocks=512)
    assert call(None) == mbd.MBD_EINVAL
    for name in ("q", "start", "lens", "table", "out"):
        assert call(a, **{name: None}) == mbd.MBD_EINVAL
        assert call(a, **{name: P + 2}) == mbd.MBD_EALIGN
    assert call(a, lse=P + 2) == mbd.MBD_EALIGN
    need = ctypes.c_uint64()
    assert L.mbd_kv_attn_workspace_bytes(ctypes.byref(c), 8, 2, 1, 512, ctypes.byref(need)) == mbd.MBD_OK and need.value > 0
    assert call(a, ws=None) == call(a, size=need.value - 1) == mbd.MBD_EINVAL
    assert call(a, ws=P + 8) == mbd.MBD_EALIGN
    assert call(_args(T=0), q=None, out=None, ws=None, size=0) == mbd.MBD_OK      # nothing to do, nothing enqueued


def test_workspace_sizes(L):
    need = ctypes.c_uint64()
    c = _cache(k_codes=None, v_codes=None, k_scale=None, v_scale=None)              # only its shape counts
    ask = lambda *a: L.mbd_kv_attn_workspace_bytes(ctypes.byref(c), *a, ctypes.byref(need))
    assert L.mbd_kv_attn_workspace_bytes(ctypes.byref(c), 8, 2, 1, 512, None) == mbd.MBD_EINVAL
    assert L.mbd_kv_attn_workspace_bytes(None, 8, 2, 1, 512, ctypes.byref(need)) == mbd.MBD_EINVAL
    assert ask(8, 2, 0, 512) == ask(9, 2, 1, 512) == ask(8, 0, 1, 512) == ask(8, 2, 1, 0) == mbd.MBD_ESHAPE
    assert ask(8, 2, 1, 1) == mbd.MBD_OK and need.value == 0                        # 16 tokens: never split
    assert ask(8, 4096, 1, 32768) == mbd.MBD_OK and 0 < need.value < 1 << 30
    assert ask(8, 64, 8192, 32768) == mbd.MBD_OK and need.value < 1 << 27           # does not grow with the rows
    assert ask(8, 1, 1 << 21, 1 << 20) == mbd.MBD_OK and need.value < 1 << 27


def test_binding_checks():
    codes = torch.zeros((4, 2, 16 * 128), dtype=torch.uint8)
    scale = torch.zeros((4, 2))
    with pytest.raises(ValueError, match="current GPU"):
        mbd.KvCache(mbd.MBD_KV_INT8, 16, 128, codes, codes, scale, scale)
    with pytest.raises(ValueError, match="block_size"):
        mbd.KvCache(mbd.MBD_KV_INT8, 32, 128, codes, codes, scale, scale)
    with pytest.raises(ValueError, match="contiguous"):
        mbd.KvCache(mbd.MBD_KV_INT8, 16, 128, codes, codes, scale, scale.double())
    with pytest.raises(ValueError, match="current GPU"):
        mbd.KvPool(16, torch.zeros((2, 4), dtype=torch.int32), torch.zeros(9, dtype=torch.int32))
    with pytest.raises(ValueError, match="n_seqs"):
        mbd.KvPool(16, torch.zeros(4, dtype=torch.int32), torch.zeros(9, dtype=torch.int32))


def test_packed_attention_arguments():
    """The bytes that the binding packs are an mbd_kv_attn_args."""
    vals = (8, 2, 4, 2, 1, 3, 0.5, 2.0, 0x1230, 1024, 2048)
    raw = mbd._ATTN_ARGS.pack(*vals)
    a = mbd.MbdKvAttnArgs.from_buffer_copy(raw)
    assert len(raw) == ctypes.sizeof(mbd.MbdKvAttnArgs)
    assert tuple(getattr(a, n) for n, _ in mbd.MbdKvAttnArgs._fields_) == vals


class _On(torch.Tensor):
    """A CPU tensor that says it is on a GPU; its memory is never reached."""
    gpu = 0

    def get_device(self):
        return self.gpu


def _on(gpu, shape, dtype=torch.int32):
    t = torch.zeros(shape, dtype=dtype).as_subclass(_On)
    t.gpu = gpu
    return t


def test_cache_and_pool_of_another_gpu(monkeypatch):
    """A cache or a pool built on GPU 0 is refused with GPU 1 current, before the library is called."""
    current = [0]
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])

    def cache(gpu):
        current[0] = gpu
        codes, scale = _on(gpu, (4, 2, 16 * 64), torch.uint8), _on(gpu, (4, 2), torch.float32)
        return mbd.KvCache(mbd.MBD_KV_INT8, 16, 64, codes, codes, scale, scale)

    def pool(gpu):
        current[0] = gpu
        return mbd.KvPool(16, _on(gpu, (2, 4)), _on(gpu, 9))

    here, other, tables = cache(1), cache(0), pool(0)
    current[0] = 1

    def no_library():
        raise AssertionError("the library was called")

    monkeypatch.setattr(mbd, "lib", no_library)
    x, ints = _on(1, (3, 2, 64), torch.bfloat16), lambda *n: _on(1, n)
    calls = {
        "append": lambda c: mbd.mbd_kv_append(c, x, x, ints(3), stream=0),
        "gather": lambda c: mbd.mbd_kv_gather(c, ints(3), x, x, stream=0),
        "attn": lambda c: mbd.mbd_kv_attn(c, x, ints(3), ints(2), ints(2, 4), x, stream=0),
    }
    for name, call in calls.items():
        with pytest.raises(ValueError, match="the cache is on"):
            call(other)
        with pytest.raises(AssertionError, match="library was called"):
            call(here)                                   # the same call with a cache of its GPU goes through
    slots = lambda p: mbd.mbd_kv_slots(p, ints(2), ints(2), ints(2), ints(1), ints(3), ints(5), None, ints(2), ints(2), ints(1), ints(2), stream=0)
    with pytest.raises(ValueError, match="the pool is on"):
        slots(tables)
    own = pool(1)
    with pytest.raises(AssertionError, match="library was called"):
        slots(own)


def test_scale_over_cap_out_of_range(L):
    """|scale| / softcap above 2^126, where fp32 cannot hold the factor of a score, is refused; the largest below is not."""
    call = lambda scale, cap: L.mbd_kv_attn(ctypes.byref(_cache()), ctypes.byref(_args(scale=scale, softcap=cap, T=0)), None, P, P, P, None, None,
                                            None, 0, None)
    for scale, cap in ((2.0 ** 64, 2.0 ** -64), (-2.0 ** 64, 2.0 ** -63), (2.0 ** 63, 2.0 ** -64)):
        assert call(scale, cap) == mbd.MBD_EINVAL
    for scale, cap in ((2.0 ** 64, 2.0 ** -62), (-2.0 ** 62, 2.0 ** -64), (0.0, 2.0 ** -64), (2.0 ** 64, 0.0), (2.0 ** -64, 2.0 ** 64)):
        assert call(scale, cap) == mbd.MBD_OK


def test_workspace_for_the_largest_step_serves_all(L):
    """A workspace made for the most requests, tokens and blocks is enough for every smaller call."""
    def size(c, *a):
        need = ctypes.c_uint64()
        assert L.mbd_kv_attn_workspace_bytes(ctypes.byref(c), *a, ctypes.byref(need)) == mbd.MBD_OK
        return need.value

    grew = 0
    for heads, group, dim in ((8, 4, 128), (1, 1, 64), (2, 16, 256), (16, 1, 192), (4, 17, 64), (128, 1, 128), (1100, 2, 64)):
        c = _cache(n_heads=heads, head_dim=dim, block_size=64)
        steps = [(n, new, cols) for n in (1, 2, 7, 16, 17, 40, 65, 130, 200, 257, 1000, 1025, 4096) for new in (1, 2, 4, 5, 9, 16, 17, 64, 300)
                 for cols in (1, 2, 5, 128, 3000)]
        sizes = {s: size(c, heads * group, *s) for s in steps}
        for big, most in sizes.items():
            for small, need in sizes.items():
                if all(a <= b for a, b in zip(small, big)):
                    assert need <= most, (heads, group, dim, small, need, big, most)
                    grew += need < most
    assert grew
