"""Refusals of the 4-bit cache and of the append with rotation: each with its status, before any GPU
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
    d = dict(fmt=mbd.MBD_KV_MXFP4, block_size=16, n_heads=2, head_dim=128, n_blocks=8, k_codes=P, v_codes=P, k_scale=P, v_scale=P)
    return mbd.MbdKvCache(**(d | kw))


def _rope(**kw):
    d = dict(table=P, n_positions=64, rot_dim=128, interleaved=0, n_q_heads=8, q=P, q_out=2 * P, q_stride=1024, q_out_stride=1024)
    return mbd.MbdRope(**(d | kw))


def _args(**kw):
    d = dict(n_heads=8, n_seqs=2, max_blocks=4, T=2, max_new=1, window=0, scale=0.1, softcap=0.0, slopes=None, q_stride=1024, out_stride=1024)
    return mbd.MbdKvAttnArgs(**(d | kw))


BAD_CACHES = [(dict(fmt=4), "EINVAL"), (dict(block_size=8), "ESHAPE"), (dict(block_size=48), "ESHAPE"), (dict(head_dim=96), "ESHAPE"),
              (dict(head_dim=32), "ESHAPE"), (dict(head_dim=512), "ESHAPE"), (dict(n_heads=0), "ESHAPE"), (dict(n_heads=65536), "ESHAPE"),
              (dict(n_blocks=0), "ESHAPE"), (dict(n_blocks=1 << 27), "ESHAPE"), (dict(k_codes=None), "EINVAL"), (dict(k_scale=None), "EINVAL"),
              (dict(v_codes=P + 8), "EALIGN"), (dict(v_scale=P + 2), "EALIGN")]


@pytest.mark.parametrize("change,status", BAD_CACHES)
def test_bad_caches(L, change, status):
    want = getattr(mbd, "MBD_" + status)
    c = ctypes.byref(_cache(**change))
    assert L.mbd_kv_append(c, P, P, mbd.MBD_BF16, 256, 256, P, 1, None) == want
    assert L.mbd_kv_append_rope(c, ctypes.byref(_rope()), P, P, mbd.MBD_BF16, 256, 256, P, P, 1, None) == want
    assert L.mbd_kv_gather(c, P, 1, mbd.MBD_F32, P, P, None) == want
    assert L.mbd_kv_attn(c, ctypes.byref(_args()), P, P, P, P, P, None, P, 1 << 30, None) == want
    assert L.mbd_last_error()


@pytest.mark.parametrize("fmt", ["MBD_KV_MXFP4", "MBD_KV_INT8", "MBD_KV_E4M3"])
def test_append_rope_arguments(L, fmt):
    c = ctypes.byref(_cache(fmt=getattr(mbd, fmt)))

    def app(k=P, v=P, dt=mbd.MBD_BF16, ks=256, vs=256, s=P, pos=P, T=1, rope=True, **kw):
        return L.mbd_kv_append_rope(c, ctypes.byref(_rope(**kw)) if rope else None, k, v, dt, ks, vs, s, pos, T, None)

    assert L.mbd_kv_append_rope(None, ctypes.byref(_rope()), P, P, 1, 256, 256, P, P, 1, None) == mbd.MBD_EINVAL
    assert app(k=None) == app(v=None) == app(s=None) == app(pos=None) == app(dt=3) == app(rope=False) == mbd.MBD_EINVAL
    assert app(k=P + 8) == app(v=P + 4) == app(s=P + 1) == app(pos=P + 2) == mbd.MBD_EALIGN
    assert app(ks=248) == app(vs=260) == app(T=-1) == app(T=(1 << 24) + 1) == mbd.MBD_ESHAPE
    assert app(table=None) == app(q=None) == app(q_out=None) == app(q_out=P) == mbd.MBD_EINVAL
    assert app(table=P + 8) == app(q=P + 8) == app(q_out=P + 4) == mbd.MBD_EALIGN
    for rot in (0, -8, 4, 12, 136, 256):
        assert app(rot_dim=rot) == mbd.MBD_ESHAPE, rot
    assert app(n_positions=0) == app(n_positions=-5) == app(n_q_heads=-1) == app(n_q_heads=65536) == mbd.MBD_ESHAPE
    assert app(q_stride=1016) == app(q_out_stride=1028) == mbd.MBD_ESHAPE
    # nothing to do, nothing enqueued; without queries theirs are not looked at
    assert app(T=0, k=None, v=None, s=None, pos=None, q=None, q_out=None) == mbd.MBD_OK
    assert app(T=0, n_q_heads=0, q=P + 2, q_stride=1) == mbd.MBD_OK
    assert app(T=0, rot_dim=7) == mbd.MBD_ESHAPE
    most = dict(n_q_heads=1 << 10, q_stride=1 << 17, q_out_stride=1 << 17)
    assert app(T=1 << 24, **most) == app(T=1 << 21, **most) == app(T=1 << 19, **most) == mbd.MBD_ESHAPE      # 2^36 elements of queries


def test_attention_arguments(L):
    c = ctypes.byref(_cache())
    call = lambda **kw: L.mbd_kv_attn(c, ctypes.byref(_args(**kw)), P, P, P, P, P, None, P, 1 << 40, None)
    for kw, status in ((dict(n_heads=7), "ESHAPE"), (dict(max_new=0), "ESHAPE"), (dict(window=-1), "EINVAL"), (dict(scale=float("nan")), "EINVAL"),
                       (dict(softcap=-1.0), "EINVAL"), (dict(scale=2.0 ** 64, softcap=2.0 ** -64), "EINVAL"), (dict(q_stride=1016), "ESHAPE")):
        assert call(**kw) == getattr(mbd, "MBD_" + status), kw
    for name in ("q", "start", "lens", "table", "out"):
        d = dict(q=P, start=P, lens=P, table=P, out=P)
        for bad, status in ((None, mbd.MBD_EINVAL), (P + 2, mbd.MBD_EALIGN)):
            p = d | {name: bad}
            assert L.mbd_kv_attn(c, ctypes.byref(_args()), p["q"], p["start"], p["lens"], p["table"], p["out"], None, P, 1 << 40, None) == status
    need = ctypes.c_uint64()
    assert L.mbd_kv_attn_workspace_bytes(c, 8, 2, 1, 512, ctypes.byref(need)) == mbd.MBD_OK and need.value > 0
    long = ctypes.byref(_args(max_blocks=512))
    assert L.mbd_kv_attn(c, long, P, P, P, P, P, None, None, 0, None) == mbd.MBD_EINVAL
    assert L.mbd_kv_attn(c, long, P, P, P, P, P, None, P, need.value - 1, None) == mbd.MBD_EINVAL
    assert L.mbd_kv_attn(c, long, P, P, P, P, P, None, P + 8, need.value, None) == mbd.MBD_EALIGN
    assert L.mbd_kv_attn(c, ctypes.byref(_args(T=0)), None, P, P, P, None, None, None, 0, None) == mbd.MBD_OK


def test_workspace_for_the_largest_step_serves_all(L):
    """A workspace made for the most requests, tokens and blocks is enough for every smaller call."""
    def size(c, *a):
        need = ctypes.c_uint64()
        assert L.mbd_kv_attn_workspace_bytes(ctypes.byref(c), *a, ctypes.byref(need)) == mbd.MBD_OK
        return need.value

    for heads, group, dim in ((8, 4, 128), (1, 1, 64), (2, 16, 256), (16, 1, 192), (4, 17, 64), (1100, 2, 64)):
        c = _cache(n_heads=heads, head_dim=dim, block_size=64)
        steps = [(n, new, cols) for n in (1, 7, 17, 40, 130, 257, 1025, 4096) for new in (1, 2, 5, 16, 17, 33, 64, 300) for cols in (1, 2, 128, 3000)]
        sizes = {s: size(c, heads * group, *s) for s in steps}
        for big, most in sizes.items():
            for small, need in sizes.items():
                if all(a <= b for a, b in zip(small, big)):
                    assert need <= most, (heads, group, dim, small, need, big, most)


def test_binding_checks():
    codes, scale = torch.zeros((4, 2, 16 * 64), dtype=torch.uint8), torch.zeros((4, 2, 16 * 4), dtype=torch.uint8)
    with pytest.raises(ValueError, match="current GPU"):
        mbd.KvCache(mbd.MBD_KV_MXFP4, 16, 128, codes, codes, scale, scale)
    with pytest.raises(ValueError, match="head_dim / 2"):
        mbd.KvCache(mbd.MBD_KV_MXFP4, 32, 128, codes, codes, scale, scale)
    for bad in (scale.float(), scale[:, :, :32], torch.zeros((4, 2)), scale.transpose(0, 1)):
        with pytest.raises(ValueError, match="contiguous"):
            mbd.KvCache(mbd.MBD_KV_MXFP4, 16, 128, codes, codes, scale, bad)
    with pytest.raises(ValueError, match="block_size"):
        mbd.KvCache(mbd.MBD_KV_INT8, 16, 128, codes, codes, scale, scale)


def test_packed_rotation():
    """The bytes that the binding packs are an mbd_rope."""
    vals = (0x1230, 77, 64, 1, 8, 0x4560, 0x7890, 1024, 2048)
    raw = mbd._ROPE.pack(*vals)
    r = mbd.MbdRope.from_buffer_copy(raw)
    assert len(raw) == ctypes.sizeof(mbd.MbdRope)
    assert tuple(getattr(r, n) for n, _ in mbd.MbdRope._fields_) == vals


class _On(torch.Tensor):
    """A CPU tensor that says it is on a GPU; its memory is never reached."""
    gpu = 0

    def get_device(self):
        return self.gpu


def _on(gpu, shape, dtype=torch.int32):
    t = torch.zeros(shape, dtype=dtype).as_subclass(_On)
    t.gpu = gpu
    return t


def test_rope_binding_refuses(monkeypatch):
    """What the binding of the append with rotation refuses before the library is called."""
    current = [1]
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])

    def cache(gpu):
        current[0] = gpu
        codes, scale = _on(gpu, (4, 2, 16 * 32), torch.uint8), _on(gpu, (4, 2, 16 * 2), torch.uint8)
        return mbd.KvCache(mbd.MBD_KV_MXFP4, 16, 64, codes, codes, scale, scale)

    other, here = cache(0), cache(1)

    def no_library():
        raise AssertionError("the library was called")

    monkeypatch.setattr(mbd, "lib", no_library)
    x, ints, f32 = _on(1, (3, 2, 64), torch.bfloat16), lambda *n: _on(1, n), torch.float32
    q, q_out, table = _on(1, (3, 4, 64), torch.bfloat16), _on(1, (3, 4, 64), torch.bfloat16), _on(1, (9, 64), f32)

    def call(c=here, k=x, v=x, slots=ints(3), pos=ints(3), t=table, **kw):
        mbd.mbd_kv_append_rope(c, k, v, slots, pos, t, stream=0, **kw)

    with pytest.raises(AssertionError, match="library was called"):
        call(q=q, q_out=q_out)
    with pytest.raises(AssertionError, match="library was called"):
        call()
    for kw, what in ((dict(c=other), "the cache is on"), (dict(pos=ints(2)), "positions"), (dict(slots=ints(4)), "slots"), (dict(v=_on(1, (2, 2, 64), torch.bfloat16)), "as many"),
                     (dict(t=_on(0, (9, 64), f32)), "table is on"), (dict(t=table[:, ::2]), "contiguous fp32"), (dict(t=_on(1, (9, 64), torch.float64)), "fp32"),
                     (dict(q=q), "go together"), (dict(q=_on(1, (2, 4, 64), torch.bfloat16), q_out=q_out), "as many"), (dict(q=q, q_out=q_out[:, :2]), "q_out"),
                     (dict(q=q.float(), q_out=q_out), "q must"), (dict(q=q, q_out=_on(1, (3, 4, 64), f32)), "q_out"),
                     (dict(q=_on(0, (3, 4, 64), torch.bfloat16), q_out=q_out), "q is on"), (dict(q=q[..., :32], q_out=q_out), "q must")):
        with pytest.raises(ValueError, match=what):
            call(**kw)
