"""Pins of the 8-bit append's oracle where tokens are not stored."""
import numpy as np
import pytest

from oracle import kv


@pytest.mark.parametrize("fmt", [kv.INT8, kv.E4M3])
def test_unstored_tokens_leave_no_trace(fmt):
    rng = np.random.default_rng(3)
    start = rng.integers(0, 120, (3, 2, 16, 64)).astype(np.uint8)
    x = rng.standard_normal((20, 2, 64))
    slots, stored = np.concatenate([np.arange(4, 14), np.arange(16, 26)]), rng.random(20) < 0.6
    scale = np.full((3, 2), 2.0 ** -9, np.float32)
    loud = np.where(stored[:, None, None], x, 1e9)
    a, sa, b, sb = start.copy(), scale.copy(), start.copy(), scale.copy()
    kv.append(a, sa, x, slots, fmt, stored)
    kv.append(b, sb, loud, slots, fmt, stored)
    assert np.array_equal(a, b) and np.array_equal(sa, sb)
    # the stored tokens' codes and the scales are those of a call whose other tokens are zeros
    c, sc = start.copy(), scale.copy()
    kv.append(c, sc, np.where(stored[:, None, None], x, 0.0), slots, fmt)
    assert np.array_equal(sa, sc)
    for s, ok in zip(slots, stored):
        if ok:
            assert np.array_equal(a[s // 16, :, s % 16], c[s // 16, :, s % 16])
    # block 0 went on: places that are not stored hold the same values as before, to half a step of the new scale and
    # (e4m3) of themselves; block 1 began: zeros
    for s, ok in zip(slots, stored):
        if ok:
            continue
        was, now = kv.decode(start[s // 16, :, s % 16], fmt) * 2.0 ** -9, kv.decode(a[s // 16, :, s % 16], fmt) * sa[s // 16][:, None]
        step = sa[s // 16][:, None] * (1.0 if fmt == kv.INT8 else 2.0 ** -9)
        if s < 16:
            assert (np.abs(now - was) <= step / 2 + (0 if fmt == kv.INT8 else 2.0 ** -4 * np.abs(was)) + 1e-9).all()
        else:
            assert (now == 0).all()
    assert np.array_equal(a[2], start[2]) and np.array_equal(a[0, :, 14:], start[0, :, 14:])


def test_nothing_stored(fmt=kv.INT8):
    codes, scale = np.full((2, 1, 16, 64), 9, np.uint8), np.full((2, 1), 5.0, np.float32)
    kv.append(codes, scale, np.ones((4, 1, 64)), np.array([3, 4, 16, 17]), fmt, np.zeros(4, bool))
    assert (codes == 9).all() and scale.ravel().tolist() == [5.0, 0.0]          # a block that begins has no scale yet
