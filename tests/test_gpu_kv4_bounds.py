"""Attention over the 4-bit KV cache within bounds derived row by row: outputs by the rounding of their type and fp32
sums alone, scores by the roundings of fp32."""
import numpy as np
import pytest

from oracle import kv, kv4
from tests.test_gpu_kv4 import Cache, _ints, _mbd, dev  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def _attend(dev, dim, bs, hkv, group, lens, new, fill, queries, width=None, max_new=None, **opts):  # noqa: F811
    """One call; returns its outputs, and the oracle's arguments."""
    mbd = _mbd()
    lens, new = np.array(lens), np.array(new)
    n, hq = len(lens), hkv * group
    held = -(-lens // bs)
    blocks = int(held.sum()) + 2
    c = Cache(blocks, hkv, dim, bs, dev, seed=dim + n)
    order, at = c.rng.permutation(blocks), 0
    table = np.full((n, width or max(1, int(held.max()))), -1)
    for i in range(n):
        table[i, :held[i]] = order[at:at + held[i]]
        at += held[i]
    fill(c, order[:at])
    for i in range(n):
        if lens[i] % bs:
            c.spoil(table[i, lens[i] // bs], lens[i] % bs)
    start = np.concatenate([[0], np.cumsum(new)])
    T, most = int(start[-1]), max_new or int(new.max())
    q = torch.from_numpy(queries(c.rng, (T, hq, dim))).to(torch.bfloat16)
    cache = c.device()
    out, lse = torch.zeros((T, hq, dim), dtype=torch.bfloat16, device=dev), torch.zeros((T, hq), device=dev)
    ws = torch.full((max(16, mbd.mbd_kv_attn_workspace_bytes(cache, hq, n, most, table.shape[1])),), 0xFF, dtype=torch.uint8, device=dev)
    mbd.mbd_kv_attn(cache, q.to(dev), _ints(start, dev), _ints(lens, dev), _ints(table, dev), out, ws, max_new=most, lse=lse, **opts)
    torch.cuda.synchronize()
    k, v = c.values()
    one = np.ones(k.shape[:2])
    args = [q.double().numpy(), start, lens, table, k, v, one, one, bs, opts["scale"], opts.get("softcap", 0.0), opts.get("window", 0)]
    return out.double().cpu().numpy(), lse.double().cpu().numpy(), args


def _normal(c, blocks):
    c.fill(blocks)


# lengths, new tokens, KV heads, query heads each, columns of the table (None: as many as needed)
SHAPES = [([3, 40, 333], [1, 1, 1], 2, 4, None),                 # a workgroup a request
          ([3, 40, 333, 2500], [1, 3, 1, 2], 2, 4, None),        # parts of four waves, joined
          ([5, 60, 900, 17], [1, 2, 40, 17], 1, 3, None),        # two row tiles
          ([9, 70, 33, 120] * 18, [1] * 72, 16, 1, 300)]         # parts of one wave


@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("lens,new,hkv,group,width", SHAPES)
@pytest.mark.parametrize("opts", [{}, dict(softcap=4.0, window=200)])
def test_outputs_are_off_by_their_own_rounding(dev, dim, lens, new, hkv, group, width, opts):  # noqa: F811
    """Scores near each other, so that every token has a weight that no short type holds."""
    scale = 0.05 * dim ** -0.5
    o, lse, args = _attend(dev, dim, 16, hkv, group, lens, new, _normal, lambda rng, s: rng.standard_normal(s), width, scale=scale, **opts)
    ref, ref_lse, mine = kv.attention(*args)
    assert mine.all()
    q, k, v = args[0], args[4], args[5]
    args[5] = np.abs(v)
    weight, _, _ = kv.attention(*args)                           # sum_j w_j |v_j|
    # A score is a sum of dim products, exact, in fp32, a step of the largest partial sum lost at each addition at most; A bounds
    # that sum: |q_d| times the head's largest |k_d|.  Behind it the factor and the product with it, half a step of the score each (with the
    # cap a quotient, an exponential, a reciprocal and a product more, of a value below it: four steps and a step each).
    kmax = np.repeat(np.abs(k).max((0, 2)), group, 0)[None]
    A = scale * (np.abs(q) * kmax).sum(-1)
    du = 2.0 ** -23 * (dim + 4) * A + (2.0 ** -20 * opts["softcap"] if opts else 0.0)
    # A weight is off by du, by its exponent's rounding (scores are below 2^4: 2^-20) and its exponential's (2^-23), and in
    # the product by what two bf16 leave of it: 2^-8 of 2^-8.  The sum of weights is off by the first three; both by fp32 sums of
    # twice as many products as a row has tokens, a step of the whole each at most, and over waves and parts.
    assert A.max() < 2 ** 4
    sums = 2.0 ** -23 * (2 * np.repeat(lens, new)[:, None] + 64)
    tol = 2.0 ** -8 * np.abs(ref) + 1.01 * (2.0 ** -16 + 2 * (du + 2.0 ** -19) + 2 * sums)[..., None] * weight
    over = np.abs(o - ref) - tol
    assert (over <= 0).all(), "worst %.3g over, of |o| %.3g and weight %.3g" % (
        over.max(), np.abs(ref).flat[over.argmax()], weight.flat[over.argmax()])
    # the logarithm of the sum moves by as much as the scores and the sum of weights do, and is rounded itself
    assert (np.abs(lse - ref_lse) <= du + sums + 2.0 ** -19 + 2.0 ** -22 * np.abs(ref_lse)).all()


@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("rows", [1, 5, 40])                     # query heads: one row tile and two
@pytest.mark.parametrize("window", [0, 1])
def test_scores_keep_every_bit_of_fp32(dev, dim, rows, window):  # noqa: F811
    """In each group one product of 0.5 to 6 among products of 2^-16 to 2^-5, all of them multiples of 2^-16 and below 2^6 when
    added up: exact in fp32 in any order, while a sum that drops what lies 17 bits below its largest term loses some 2^-9.  A row
    sees one token, so the log-sum-exp is its score."""
    hkv, lens = 2, [1, 200] if window else [1, 1]

    def fill(c, blocks):
        c.fill(blocks)
        c.k[blocks] = c.rng.integers(1, 8, c.k[blocks].shape)    # all positive
        c.ke[blocks] = 127

    def queries(rng, shape):
        q = rng.integers(1, 128, shape) * 2.0 ** -15
        q[..., ::32] = 1.0
        return q

    o, lse, args = _attend(dev, dim, 16, hkv, rows, lens, [1, 1], fill, queries, scale=1.0, window=window)
    ref, ref_lse, mine = kv.attention(*args)
    assert mine.all() and np.array_equal(ref_lse * 2 ** 16, np.rint(ref_lse * 2 ** 16)) and (ref_lse < 2 ** 6).all()
    # log2(e) as fp32, the score times it, the sum of base and weight's logarithm, ln 2 as fp32 and the product with it: half a step
    # (2^-24) each; the weight that the fused exponent leaves, and its logarithm: a step (2^-23) each
    assert (np.abs(lse - ref_lse) <= 5 * 2.0 ** -24 * ref_lse + 2 * 2.0 ** -23).all()
    np.testing.assert_array_equal(o, np.repeat(np.stack([args[5][args[3][i, (n - 1) // 16], :, (n - 1) % 16] for i, n in enumerate(lens)]), rows, 1))


@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("lens,new,hkv,group,width", SHAPES)
@pytest.mark.parametrize("opts", [{}, dict(window=200)])
def test_large_scores_within_their_roundings(dev, dim, lens, new, hkv, group, width, opts):  # noqa: F811
    """Scores up to some hundreds, maxima that move late, weights that underflow.  Queries are whole numbers, so every product q k is
    one of 2^-3 and below 2^14 when added up: exact in fp32 in any order."""
    scale = 2.0
    o, lse, args = _attend(dev, dim, 16, hkv, group, lens, new, _normal, lambda rng, s: rng.integers(-3, 4, s).astype(float), width, scale=scale, **opts)
    ref, ref_lse, mine = kv.attention(*args)
    q, start, table, k, v = args[0], args[1], args[3], args[4], args[5]
    args[5] = np.abs(v)
    weight, _, _ = kv.attention(*args)
    U = np.zeros(lse.shape)                                      # a row's largest |score|
    for i, n in enumerate(lens):
        j = np.arange(n)
        for h in range(hkv):
            u = q[start[i]:start[i + 1], h * group:(h + 1) * group] @ k[table[i][j // 16], h, j % 16].T
            U[start[i]:start[i + 1], h * group:(h + 1) * group] = scale * np.abs(u).max(-1)
    assert mine.all() and U.max() > 100 and 6 * 3 * dim < 2 ** 14
    # log2(e) times the scale as fp32 (its own error and a rounding), the product with it, its difference to the base (twice as
    # large at most); for the log-sum-exp the sum with the base, ln 2 and the product with it: eight half steps of the score.
    du = 8 * 2.0 ** -24 * U
    sums = 2.0 ** -23 * (2 * np.repeat(lens, new)[:, None] + 64)
    tol = 2.0 ** -8 * np.abs(ref) + 1.01 * (2.0 ** -16 + 2 * (du + 2.0 ** -22) + 2 * sums)[..., None] * weight + 2.0 ** -100
    over = np.abs(o - ref) - tol
    assert (over <= 0).all(), "worst %.3g over, of |o| %.3g and weight %.3g" % (
        over.max(), np.abs(ref).flat[over.argmax()], weight.flat[over.argmax()])
    assert (np.abs(lse - ref_lse) <= du + sums + 2.0 ** -22).all()


@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("last", [1, 15, 16, 17, 31, 32])
def test_rows_of_the_last_row_tile(dev, dim, last):  # noqa: F811
    """Prompts whose query rows leave 1 to 32 in the last tile of 32, whole, and cut behind 3000 tokens."""
    test_outputs_are_off_by_their_own_rounding(dev, dim, [32 + last, 3000 + last], [32 + last, last if last > 16 else 32 + last], 2, 1, None, {})
    if (64 + last) % 3 == 0:
        test_outputs_are_off_by_their_own_rounding(dev, dim, [2100, 22], [(64 + last) // 3, 1], 1, 3, None, dict(softcap=4.0, window=1700))
