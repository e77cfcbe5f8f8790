"""Pins of the 4-bit KV-cache oracle: the documented layout, codes and exponents by brute force, and
the rotation against complex multiplication."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import kv4


@pytest.mark.parametrize("bs,dim", [(16, 64), (32, 128), (64, 192), (256, 256)])
def test_layouts_are_permutations(bs, dim):
    rng = np.random.default_rng(0)
    for values in (False, True):
        byte, half = kv4._order(bs, dim, values)
        assert np.array_equal(np.sort((2 * byte + half).ravel()), np.arange(bs * dim))
        raw = rng.integers(0, 256, (2, 3, bs * dim // 2)).astype(np.uint8)
        assert np.array_equal(kv4.pack(kv4.unpack(raw, bs, dim, values), values), raw)
    assert np.array_equal(np.sort(kv4._scale_order(bs, dim).ravel()), np.arange(bs * dim // 32))
    raw = rng.integers(0, 256, (2, 3, bs * dim // 32)).astype(np.uint8)
    assert np.array_equal(kv4.pack_scales(kv4.unpack_scales(raw, bs, dim)), raw)


def test_layout_by_hand():
    # a key lane's 16 bytes: 32 channels of one token; a value lane's: 4 tokens x 8 channels, or 4 x 4 in a half slab
    assert [kv4.code_at(21, d, 192, False) for d in (64, 65, 94, 95)] == [(1536 + 512 + 80, 0), (1536 + 512 + 80, 1), (1536 + 512 + 95, 0), (1536 + 512 + 95, 1)]
    assert [kv4.code_at(6, d, 192, True)[0] for d in (16, 23, 127)] == [256 + 32 + 8, 256 + 32 + 8 + 3, 256 + 240 + 8 + 3]
    assert [kv4.code_at(6, d, 192, True)[0] for d in (128, 131, 132, 191)] == [1024 + 128 + 4, 1024 + 128 + 5, 1024 + 128 + 12, 1024 + 128 + 120 + 5]
    assert kv4.scale_at(18, 3, 128) == 64 + 48 + 2


def test_codes_are_the_nearest():
    exact = [Fraction(float(v)) for v in kv4.VALUES]
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.uniform(-8, 8, 3000), [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 6.99, 7.0], [0.0, -0.0, -0.2]])
    codes = kv4.encode(x)
    for v, c in zip(x, codes):
        off = [abs(min(abs(Fraction(float(v))), Fraction(6)) - e) for e in exact]
        best = [i for i, o in enumerate(off) if o == min(off)]
        want = best[0] if len(best) == 1 else next(i for i in best if i % 2 == 0)
        assert c == want + 8 * bool(np.signbit(v))
    assert kv4.encode(np.array([np.inf, -np.inf, np.nan, -np.nan])).tolist() == [7, 15, 0, 0]
    assert kv4.decode(np.arange(16)).tolist() == [0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6]


def test_exponents():
    for amax, e in ((0, -100), (1e-45, -100), (7.0, 0), (np.nextafter(np.float32(7), np.float32(9)), 1), (3.5, -1), (6.0, 0), (2.0 ** 60 * 7, 60),
                    (np.finfo(np.float32).max, 125), (7 * 2.0 ** -100, -100), (7.01 * 2.0 ** -100, -99)):
        assert kv4.exponent(float(amax)) == e, amax
    # no value is off by more than half the largest step, 2^e, and the smaller ones by half of theirs
    x = np.random.default_rng(2).standard_normal((500, 64)) * 3
    codes, exps = kv4.quantise(x)
    unit = np.repeat(2.0 ** (exps.astype(float) - 127), 32, 1)
    assert (np.abs(kv4.values(codes, exps) - x) <= unit * np.where(np.abs(x) > 4 * unit, 1.0, np.where(np.abs(x) > 2 * unit, 0.5, 0.25))).all()


def test_turn_is_a_complex_product():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((4, 2, 64)).astype(np.float32)
    angle = rng.uniform(0, 6, (9, 16))
    table = np.float32(np.concatenate([np.cos(angle), np.sin(angle)], 1))
    at = [3, 8, -1, 9]
    for pairs in (False, True):
        out = kv4.turn(x, table, at, pairs)
        np.testing.assert_array_equal(out[2:], x[2:])
        np.testing.assert_array_equal(out[..., 32:], x[..., 32:])
        for t in (0, 1):
            a, b = (x[t, :, 0:32:2], x[t, :, 1:32:2]) if pairs else (x[t, :, :16], x[t, :, 16:32])
            z = (a + 1j * b) * np.exp(1j * angle[at[t]])
            got = out[t, :, 0:32:2] + 1j * out[t, :, 1:32:2] if pairs else out[t, :, :16] + 1j * out[t, :, 16:32]
            np.testing.assert_allclose(got, z, atol=2.0 ** -21)      # four fp32 roundings of values below 2^2
            np.testing.assert_array_equal(out.astype(np.float32).astype(np.float64), out)
