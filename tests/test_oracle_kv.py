"""Pins of the KV-cache oracle: the documented byte order, 8-bit codes, the append's
scale rule, the bookkeeping, and attention against a second formulation."""
import numpy as np
import pytest

from oracle import kv

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("bs,dim", [(16, 64), (32, 128), (64, 192), (256, 256)])
def test_byte_orders_are_permutations(bs, dim):
    for values in (False, True):
        at = kv.byte_order(bs, dim, values)
        assert np.array_equal(np.sort(at.ravel()), np.arange(bs * dim))
        raw = np.random.default_rng(0).integers(0, 256, (2, 3, bs * dim)).astype(np.uint8)
        assert np.array_equal(kv.pack(kv.unpack(raw, bs, dim, values), values), raw)
    # lane (g, m) of slab s: 16 bytes of one token's channels; 4 tokens x 4 channels
    k, v = kv.byte_order(bs, dim, False), kv.byte_order(bs, dim, True)
    assert np.array_equal(k[3, 16:32], 256 + 48 + np.arange(16))
    assert np.array_equal(v[4:8, 8:12].T.ravel(), 256 + 32 + np.arange(16))


def test_e4m3_codes_match_torch():
    every = torch.arange(256, dtype=torch.uint8)
    want = every.view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(kv.decode(every.numpy(), kv.E4M3), want)
    rng = np.random.default_rng(1)
    mids = (kv._E4M3[1:] + kv._E4M3[:-1]) / 2                    # exact ties
    x = np.concatenate([rng.standard_normal(5000) * 100, mids, -mids, kv._E4M3, [0.0, -0.0]]).astype(np.float32)
    x = x[np.abs(x) <= 448]
    got = kv.encode(x.astype(np.float64), kv.E4M3)
    np.testing.assert_array_equal(got, torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    assert kv.encode(np.array([1e9, -np.inf, np.nan]), kv.E4M3).tolist() == [126, 254, 0]


def test_int8_codes():
    assert kv.encode(np.array([0.5, 1.5, -2.5, 126.6, 127.49, 300, -300, np.inf, np.nan]), kv.INT8).astype(np.int8).tolist() == \
        [0, 2, -2, 127, 127, 127, -127, 127, 0]
    assert kv.decode(np.arange(256).astype(np.uint8), kv.INT8).tolist() == list(np.arange(256).astype(np.uint8).view(np.int8))


def test_wanted_scales():
    assert kv.wanted_scale(0, kv.E4M3) == kv.wanted_scale(0, kv.INT8) == 0
    for amax, s in ((448.0, 1.0), (np.nextafter(np.float32(448), np.float32(1e9)), 2.0), (224.0, 0.5), (1e-45, 2.0 ** -126)):
        assert kv.wanted_scale(amax, kv.E4M3) == s
    assert abs(kv.wanted_scale(127.0, kv.INT8) - 1) < 2.0 ** -22


@pytest.mark.parametrize("fmt", [kv.INT8, kv.E4M3])
def test_append_error_stays_near_one_rounding(fmt):
    """Token by token into one block with rising magnitudes: each re-scaling adds at most
    half a step of the scale then in force, and scales only rise."""
    rng = np.random.default_rng(2)
    x = rng.standard_normal((16, 1, 64)) * np.linspace(0.1, 1.5, 16)[:, None, None]
    codes, scale = np.full((1, 1, 16, 64), 0xFF, np.uint8), np.full((1, 1), np.nan, np.float32)
    scales = []
    for t in range(16):
        kv.append(codes, scale, x[t:t + 1], [t], fmt)
        scales.append(float(scale[0, 0]))
    assert scales == sorted(scales)
    err = np.abs(kv.decode(codes, fmt)[0, 0] * scales[-1] - x[:, 0])
    grew = 1 + sum(b > a for a, b in zip(scales, scales[1:]))
    step = scales[-1] if fmt == kv.INT8 else np.maximum(np.abs(x[:, 0]) * 2.0 ** -3, scales[-1] * 2.0 ** -9)
    assert (err <= 0.5 * step * (grew if fmt == kv.INT8 else 1.01) * 1.001).all()


def test_slots_by_hand():
    # blocks of 16; request 0 ends and returns 7, 8; request 1 crosses a block; request 2 is a prompt that finds none left
    table = np.array([[7, 8, -1, -1], [3, -1, -1, -1], [-1, -1, -1, -1], [5, -1, -1, -1]])
    free = np.array([1, -9, -9, -9, -9])
    got = kv.slots([-1, 2, 33, 1], [20, 15, 0, 3], [2, 1, 0, 1], table, free, 1, 16, 40)
    assert got["status"].tolist() == [0, 0, 1, 0]
    assert got["seq_start"].tolist() == [0, 0, 2, 35, 36]
    assert table[1].tolist() == [3, 8, -1, -1] and table[2].tolist() == [-1] * 4
    assert got["slots"][:2].tolist() == [3 * 16 + 15, 8 * 16] and got["slots"][35] == 5 * 16 + 3
    assert (got["slots"][2:35] == -1).all() and (got["slots"][36:] == -1).all()
    assert got["lens_out"].tolist() == [0, 17, 0, 4] and got["held_out"].tolist() == [0, 2, 0, 1]
    assert got["n_free_out"] == 2 and free[:2].tolist() == [1, 7]


def test_attention_against_softmax():
    rng = np.random.default_rng(3)
    bs, dim, heads = 16, 64, 4
    k, v = rng.integers(-127, 128, (5, 2, bs, dim)).astype(float), rng.integers(-127, 128, (5, 2, bs, dim)).astype(float)
    ks, vs = rng.random((5, 2)).astype(np.float32) / 60, rng.random((5, 2)).astype(np.float32)
    table = np.array([[4, 0, 2], [1, 3, -1]])
    q = rng.standard_normal((5, heads, dim))
    o, lse, mine = kv.attention(q, [0, 3, 4], [37, 20], table, k, v, ks, vs, bs, 0.1)
    assert mine.tolist() == [True] * 4 + [False] and not o[4].any()
    kk = torch.tensor(k * ks[..., None, None])[table[0]].permute(1, 0, 2, 3).reshape(2, 48, dim)[:, :37]
    vv = torch.tensor(v * vs[..., None, None])[table[0]].permute(1, 0, 2, 3).reshape(2, 48, dim)[:, :37]
    for r in range(3):
        see = 37 - 3 + r + 1
        for h in range(heads):
            u = kk[h // 2, :see] @ torch.tensor(q[r, h]) * 0.1
            np.testing.assert_allclose(o[r, h], (torch.softmax(u, 0) @ vv[h // 2, :see]).numpy(), rtol=1e-12, atol=1e-12)
            np.testing.assert_allclose(lse[r, h], torch.logsumexp(u, 0).item(), rtol=1e-12)
    # a request with more new tokens than cached ones has rows before its start: nothing to see
    o, lse, _ = kv.attention(q[:3], [0, 3], [1], table[:1], k, v, ks, vs, bs, 0.1)
    assert not o[:2].any() and np.isneginf(lse[:2]).all() and np.isfinite(lse[2]).all()
