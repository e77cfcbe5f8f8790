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
