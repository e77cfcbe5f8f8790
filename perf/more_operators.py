"""Measured cases of the 4-bit KV cache and of the append that turns keys and queries by their positions.

The 4-bit cache holds e2m1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) with one power of two for each 32
neighbouring channels of a token's head, kept as its exponent + 127 in a byte.  Codes lie in tiles of 16 tokens, two
to a byte (the even channel in the low half); for token t of a tile and channel d of D
    K: byte  d / 32 * 256 + t * 16 + d % 32 / 2
    V: byte  d / 128 * 1024 + t / 4 * 256 + d % 128 / 8 * 16 + t % 4 * 4 + d % 8 / 2        for d < D / 128 * 128
             d / 128 * 1024 + t / 4 * 128 + d % 64 / 4 * 8 + t % 4 * 2 + d % 4 / 2          for a last half slab
and the exponents at byte  d / 32 * 16 + t  of a tile.  The 8-bit caches are as in operators.py.
`own` false computes every operator in elementary torch operations in 32 bits, `own` true calls the library.
"""
import numpy as np
import torch

own = False

INT8, E4M3, MXFP4 = "int8", "e4m3", "mxfp4"
DEV = "cuda"
GOLDEN = 0.6180339887498949


def listed():
    return [
        # one token of one request far into its context enters one layer's cache, its queries turned too: the smallest call
        dict(name="rope 1x1 mxfp4", op="append", n=1, new_lo=1, new_hi=1, lo=30000, hi=30000, hq=32, hkv=8, d=128, bs=16, fmt=MXFP4, wide=False, rot=128, pairs=False, pad=0),
        # a decode step of a full batch, half of each head turned in neighbouring pairs
        dict(name="rope decode 64 e4m3", op="append", n=64, new_lo=1, new_hi=1, lo=0, hi=4000, hq=32, hkv=8, d=128, bs=32, fmt=E4M3, wide=False, rot=64, pairs=True, pad=0),
        # a verify step: up to 9 speculated tokens of 48 requests, fp32 projections, ragged, rows of padding behind
        dict(name="rope verify 48x9 int8", op="append", n=48, new_lo=0, new_hi=9, lo=0, hi=5000, hq=32, hkv=8, d=128, bs=32, fmt=INT8, wide=True, rot=128, pairs=False, pad=16),
        # prompts written whole
        dict(name="rope prompts mxfp4", op="append", n=13, new_lo=500, new_hi=2100, lo=0, hi=40, hq=32, hkv=8, d=128, bs=64, fmt=MXFP4, wide=False, rot=128, pairs=False, pad=0),
        # keys that are turned elsewhere, or not at all
        dict(name="append 128x4 mxfp4", op="append", n=128, new_lo=0, new_hi=4, lo=0, hi=2000, hq=0, hkv=4, d=192, bs=32, fmt=MXFP4, wide=True, rot=0, pairs=False, pad=3),
        # a whole long request read back
        dict(name="gather 32768 mxfp4", op="gather", n=32768, hkv=8, d=128, bs=64, fmt=MXFP4, wide=False),
        # one request, one token: latency
        dict(name="attn 1x2048", op="attn", n=1, new_lo=1, new_hi=1, lo=2048, hi=2048, hq=32, hkv=8, d=128, bs=16, fmt=MXFP4, softcap=0.0, window=0, alibi=False, pad=0),
        # one request with a long context
        dict(name="attn 1x100001", op="attn", n=1, new_lo=1, new_hi=1, lo=100001, hi=100001, hq=32, hkv=8, d=128, bs=64, fmt=MXFP4, softcap=0.0, window=0, alibi=False, pad=0),
        # a batch in flight, lengths from one token to 8192, one token each
        dict(name="attn 32x8192", op="attn", n=32, new_lo=1, new_hi=1, lo=1, hi=8192, hq=32, hkv=8, d=128, bs=32, fmt=MXFP4, softcap=0.0, window=0, alibi=False, pad=3),
        # a verify step of 5 tokens a request, one KV head a query head, sliding window and capped scores
        dict(name="attn verify 8x5", op="attn", n=8, new_lo=5, new_hi=5, lo=300, hi=4001, hq=16, hkv=16, d=64, bs=16, fmt=MXFP4, softcap=30.0, window=1024, alibi=False, pad=0),
        # slices of prompts behind cached prefixes
        dict(name="attn prompts 4x300", op="attn", n=4, new_lo=90, new_hi=300, lo=400, hi=2500, hq=32, hkv=8, d=128, bs=64, fmt=MXFP4, softcap=0.0, window=0, alibi=False, pad=0),
        # long contexts, 16 query heads a KV head
        dict(name="attn 32x32768", op="attn", n=32, new_lo=1, new_hi=1, lo=32768, hi=32768, hq=64, hkv=4, d=128, bs=64, fmt=MXFP4, softcap=0.0, window=0, alibi=False, pad=0),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["append", "append", "gather", "attn", "attn", "attn"])
    bs, d, hkv = rng.choice([16, 32, 64, 128]), rng.choice([64, 128, 192, 256]), rng.randint(1, 10)
    if op == "append":
        fmt = rng.choice([INT8, E4M3, MXFP4, MXFP4])
        rot = rng.choice([0, d, d, 8 * rng.randint(1, d // 8)]) if fmt == MXFP4 else rng.choice([d, d, 8 * rng.randint(1, d // 8)])
        n, hq = _log(rng, 1, 60), hkv * rng.choice([0, 1, 2, 4, 7]) if rot else 0
        hi = _log(rng, 1, max(1, 13000 // n * 8 * 128 // (hkv * d)))
        return dict(op=op, n=n, new_lo=min(hi, rng.randint(0, 2)), new_hi=hi, lo=0, hi=_log(rng, 1, 4000), hq=hq, hkv=hkv, d=d, bs=bs, fmt=fmt,
                    wide=rng.random() < 0.4, rot=rot, pairs=rng.random() < 0.4, pad=rng.randint(0, 20))
    if op == "gather":
        return dict(op=op, n=_log(rng, 1, max(1, 32768 * 8 * 128 // (hkv * d))), hkv=hkv, d=d, bs=bs, fmt=MXFP4, wide=rng.random() < 0.5)
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    if rng.random() < 0.6:
        n, new = _log(rng, 1, 64), 1
    elif rng.random() < 0.6:
        n, new = _log(rng, 1, 32), rng.randint(2, 16)
    else:
        n, new = _log(rng, 1, 4), _log(rng, 17, 300)
    hi = max(new, _log(rng, 32, max(33, min(32768, 40_000_000 // (n * hkv * group * new)))))
    if n * hi * hkv * d > 250_000_000:
        hi = max(new, 250_000_000 // (n * hkv * d))
    softcap, window, alibi = rng.choice([0.0, 0.0, 20.0]), rng.choice([0, 0, _log(rng, 1, 4096)]), rng.random() < 0.25
    return dict(op="attn", n=n, new_lo=rng.randint(1, new), new_hi=new, lo=max(new, hi // rng.choice([1, 2, 50])), hi=hi, hq=hkv * group,
                hkv=hkv, d=d, bs=bs, fmt=MXFP4, softcap=softcap, window=window, alibi=alibi, pad=rng.randint(0, 5))


# ------------------------------------------------------------------ inputs

def _spread(n, lo, hi, turn):
    """n whole numbers from hi down to lo, spread evenly: the same set for every seed."""
    return hi - np.floor((np.arange(n) * turn) % 1.0 * (hi - lo + 1)).astype(np.int64)


def _lengths(case):
    """(cached before, new) tokens of each request, before the seed orders them."""
    n = case["n"]
    new = _spread(n, case["new_lo"], case["new_hi"], 0.7548776662466927)
    before = _spread(n, case["lo"], case["hi"], GOLDEN)
    return (before if case["op"] == "append" else np.maximum(before - new, 0)), new


def _cuda(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).to(DEV)


def _paged(rng, blocks, spare):
    """Block tables of requests that hold `blocks` blocks each, from a shuffled pool; (table, blocks in the pool)."""
    total = int(blocks.sum()) + spare
    pool = rng.permutation(total)
    table = np.full((len(blocks), max(1, int(blocks.max()))), -1, np.int64)
    table[np.arange(table.shape[1])[None] < blocks[:, None]] = pool[:int(blocks.sum())]
    return table, total


def _pair_bytes():
    """Bytes of two e2m1 codes of normal values of deviation 2.2, one for each of 256 x 256 quantiles."""
    x = 2.2 * torch.special.ndtri((torch.arange(256, dtype=torch.float64) + 0.5) / 256)
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64)
    code = torch.bucketize(x.abs(), mids) + 8 * (x < 0)
    return (code[:, None] + 16 * code[None]).flatten().to(torch.uint8)


def _codes(gen, case, n_blocks):
    fmt, hkv = case["fmt"], case["hkv"]
    width = case["bs"] * case["d"] // (2 if fmt == MXFP4 else 1)
    out = torch.empty((n_blocks, hkv, width), dtype=torch.uint8, device=DEV)
    part = max(1, (1 << 26) // (hkv * width))
    pairs = _pair_bytes().to(DEV) if fmt == MXFP4 else None
    for i in range(0, n_blocks, part):
        shape = (min(part, n_blocks - i), hkv, width)
        if fmt == MXFP4:
            out[i:i + part] = pairs[torch.randint(0, 65536, shape, generator=gen, device=DEV, dtype=torch.int32)]
            continue
        x = torch.randn(shape, generator=gen, device=DEV)
        if fmt == INT8:
            out[i:i + part] = (x * 36).round_().clamp_(-127, 127).to(torch.int8).view(torch.uint8)
        else:
            out[i:i + part] = (x * 100).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return out


def _scales(gen, case, n_blocks):
    if case["fmt"] == MXFP4:
        shape = (n_blocks, case["hkv"], case["bs"] * case["d"] // 32)
        return torch.randint(125, 128, shape, generator=gen, device=DEV, dtype=torch.uint8)
    u = torch.rand((n_blocks, case["hkv"]), generator=gen, device=DEV)
    if case["fmt"] == INT8:
        return (2.6 + 1.4 * u) / 127
    return torch.where(u < 0.5, 2.0 ** -7, 2.0 ** -6)


def _cache(case, gen, n_blocks):
    s = dict(k_codes=_codes(gen, case, n_blocks), v_codes=_codes(gen, case, n_blocks), k_scale=_scales(gen, case, n_blocks),
             v_scale=_scales(gen, case, n_blocks))
    if own:
        import memory_bound_decode_amd as mbd
        fmt = {INT8: mbd.MBD_KV_INT8, E4M3: mbd.MBD_KV_E4M3, MXFP4: mbd.MBD_KV_MXFP4}[case["fmt"]]
        s["cache"] = mbd.KvCache(fmt, case["bs"], case["d"], s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"])
    return s


def prepare(case, seed):
    rng = np.random.RandomState(seed % (1 << 32))
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return {"append": _prepare_append, "gather": _prepare_gather, "attn": _prepare_attn}[case["op"]](case, rng, gen)


def _rope_table(positions, rot):
    """Cosines and sines of the angles p * 10000 ** (-2 j / rot), from 64 bits."""
    angle = torch.arange(positions, device=DEV, dtype=torch.float64)[:, None] * \
        10000.0 ** (-2.0 * torch.arange(rot // 2, device=DEV, dtype=torch.float64) / rot)
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def _prepare_append(case, rng, gen):
    bs, hq, hkv, d = case["bs"], case["hq"], case["hkv"], case["d"]
    before, new = _lengths(case)
    order = rng.permutation(case["n"])
    before, new = before[order], new[order]
    table, total = _paged(rng, -(-(before + new) // bs), 7)
    seq = np.repeat(np.arange(case["n"]), new)
    pos = np.arange(len(seq)) - np.repeat(np.cumsum(new) - new, new) + before[seq]
    slots = table[seq, pos // bs] * bs + pos % bs
    T = len(seq) + case["pad"]
    slots = np.concatenate([slots, np.full(case["pad"], -1)])
    # what the touched blocks hold afterwards, block by block
    first, last = before // bs, np.where(new > 0, (before + new - 1) // bs, before // bs - 1)
    runs = last - first + 1
    row = np.repeat(np.arange(case["n"]), runs)
    col = np.arange(len(row)) - np.repeat(np.cumsum(runs) - runs, runs) + first[row]
    touched = table[row, col]
    live = np.minimum(bs, (before + new)[row] - col * bs)
    fill = np.maximum(0, before[row] - col * bs)
    all_live = np.arange(bs)[None] < live[:, None]
    read = (touched[:, None] * bs + np.arange(bs)[None])[all_live]
    place = np.full((len(touched), bs), -1)
    block_at = np.full(total, -1)
    block_at[touched] = np.arange(len(touched))
    place[block_at[slots[:len(seq)] // bs], slots[:len(seq)] % bs] = np.arange(len(seq))
    dt = torch.float32 if case["wide"] else torch.bfloat16
    qkv = torch.randn((T, (hq + 2 * hkv) * d + 64), generator=gen, device=DEV).to(dt)      # one projection's output holds all
    q, k, v, _ = qkv.split([hq * d, hkv * d, hkv * d, 64], 1)
    s = dict(case=case, k=k.unflatten(1, (hkv, d)), v=v.unflatten(1, (hkv, d)), slots=_cuda(slots), read=_cuda(read),
             positions=_cuda(np.concatenate([pos, np.full(case["pad"], -1)])), touched=_cuda(touched, torch.int64), fill=_cuda(fill, torch.int64),
             place=_cuda(place, torch.int64), read_at=_cuda(np.flatnonzero(all_live), torch.int64),
             k_out=torch.zeros((len(read), hkv, d), device=DEV), v_out=torch.zeros((len(read), hkv, d), device=DEV))
    if case["rot"]:
        s["rope"] = _rope_table(int((before + new).max()) + 1, case["rot"])
    if hq:
        s |= dict(q=q.unflatten(1, (hq, d)), q_out=torch.zeros((T, hq, d), dtype=torch.bfloat16, device=DEV))
    return s | _cache(case, gen, total)


def _prepare_gather(case, rng, gen):
    bs = case["bs"]
    table, total = _paged(rng, np.array([-(-case["n"] // bs)]), 9)
    pos = np.arange(case["n"])
    slots = table[0, pos // bs] * bs + pos % bs
    dt = torch.float32 if case["wide"] else torch.bfloat16
    s = dict(case=case, slots=_cuda(slots), k_out=torch.zeros((case["n"], case["hkv"], case["d"]), dtype=dt, device=DEV),
             v_out=torch.zeros((case["n"], case["hkv"], case["d"]), dtype=dt, device=DEV))
    return s | _cache(case, gen, total)


def _prepare_attn(case, rng, gen):
    n, bs, hq, d = case["n"], case["bs"], case["hq"], case["d"]
    before, new = _lengths(case)
    order = rng.permutation(n)
    lens, new = (before + new)[order], new[order]
    table, total = _paged(rng, -(-lens // bs), 5)
    start = np.concatenate([[0], np.cumsum(new)])
    T = int(start[-1]) + case["pad"]
    s = dict(case=case, q=(torch.randn((T, hq, d), generator=gen, device=DEV) * 1.5).to(torch.bfloat16), table=_cuda(table), lens=_cuda(lens),
             seq_start=_cuda(start), out=torch.zeros((T, hq, d), dtype=torch.bfloat16, device=DEV), lse=torch.zeros((T, hq), device=DEV),
             scale=d ** -0.5, max_new=int(new.max()),
             slopes=torch.exp2(-8.0 * torch.arange(1, hq + 1, device=DEV) / hq) if case["alibi"] else None)
    s |= _cache(case, gen, total)
    if own:
        import memory_bound_decode_amd as mbd
        size = mbd.mbd_kv_attn_workspace_bytes(s["cache"], hq, n, s["max_new"], table.shape[1])
        s["ws"] = torch.zeros(size, dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    return {"append": _run_append, "gather": _run_gather, "attn": _run_attn}[state["case"]["op"]](state)


def _run_append(s):
    case = s["case"]
    if own:
        import memory_bound_decode_amd as mbd
        if case["rot"]:
            mbd.mbd_kv_append_rope(s["cache"], s["k"], s["v"], s["slots"], s["positions"], s["rope"], q=s.get("q"), q_out=s.get("q_out"),
                                   interleaved=case["pairs"])
        else:
            mbd.mbd_kv_append(s["cache"], s["k"], s["v"], s["slots"])
        mbd.mbd_kv_gather(s["cache"], s["read"], s["k_out"], s["v_out"])
    else:
        k, v = s["k"].float(), s["v"].float()
        if case["rot"]:
            k = _turn(s, k)
        if case["hq"]:
            known = (s["positions"] >= 0) & (s["positions"] < s["rope"].shape[0])
            s["q_out"].copy_(torch.where(known[:, None, None], _turn(s, s["q"].float()).to(torch.bfloat16), s["q_out"]))
        if case["fmt"] == MXFP4:
            _plain_append4(s, k, s["k_codes"], s["k_scale"], False, s["k_out"])
            _plain_append4(s, v, s["v_codes"], s["v_scale"], True, s["v_out"])
        else:
            _plain_append8(s, k, s["k_codes"], s["k_scale"], _k8_rows, s["k_out"])
            _plain_append8(s, v, s["v_codes"], s["v_scale"], _v8_rows, s["v_out"])
    return {k: s[k] for k in ("k_out", "v_out", "q_out") if k in s}


def _run_gather(s):
    if own:
        import memory_bound_decode_amd as mbd
        mbd.mbd_kv_gather(s["cache"], s["slots"], s["k_out"], s["v_out"])
    else:
        s["k_out"].copy_(_plain_read4(s, s["k_codes"], s["k_scale"], s["slots"].long(), False))
        s["v_out"].copy_(_plain_read4(s, s["v_codes"], s["v_scale"], s["slots"].long(), True))
    return {"k": s["k_out"], "v": s["v_out"]}


def _run_attn(s):
    if own:
        import memory_bound_decode_amd as mbd
        c = s["case"]
        mbd.mbd_kv_attn(s["cache"], s["q"], s["seq_start"], s["lens"], s["table"], s["out"], s["ws"], max_new=s["max_new"], scale=s["scale"],
                        softcap=c["softcap"], window=c["window"], slopes=s["slopes"], lse=s["lse"])
    else:
        _plain_attn(s)
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------------ plain forms

def _turn(s, x):
    """x [T, heads, d] in fp32, its first `rot` channels turned by their positions' angles; each product and sum rounded to fp32."""
    rot, half = s["case"]["rot"], s["case"]["rot"] // 2
    row = s["rope"][s["positions"].long().clamp(0, s["rope"].shape[0] - 1)][:, None]
    cos, sin = row[..., :half], row[..., half:]
    if s["case"]["pairs"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _code_values():
    half = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=DEV)
    return torch.cat([half, -half])


def _at4(case, t, values):
    """Byte offsets [tokens, d / 2] of places t of a block, for its channel pairs."""
    D = case["d"]
    d = torch.arange(0, D, 2, device=DEV)
    tile, t = (t // 16 * (8 * D))[:, None], (t % 16)[:, None]
    if not values:
        return tile + d // 32 * 256 + t * 16 + d % 32 // 2
    full = d // 128 * 1024 + t // 4 * 256 + d % 128 // 8 * 16 + t % 4 * 4 + d % 8 // 2
    half = d // 128 * 1024 + t // 4 * 128 + d % 64 // 4 * 8 + t % 4 * 2 + d % 4 // 2
    return tile + torch.where(d < D // 128 * 128, full, half)


def _scale_at4(case, t):
    return (t // 16 * (case["d"] // 2) + t % 16)[:, None] + 16 * torch.arange(case["d"] // 32, device=DEV)


def _plain_read4(s, codes, scale, slots, values):
    case = s["case"]
    block, t = slots // case["bs"], slots % case["bs"]
    head = torch.arange(case["hkv"], device=DEV)[None, :, None]
    pair = codes[block[:, None, None], head, _at4(case, t, values)[:, None]].int()
    x = _code_values()[torch.stack([pair & 15, pair >> 4], -1).flatten(-2)]
    power = scale[block[:, None, None], head, _scale_at4(case, t)[:, None]].int() - 127
    return torch.ldexp(x, power.repeat_interleave(32, 2))


def _plain_append4(s, x, codes, scale, values, out):
    case = s["case"]
    good = s["slots"] >= 0
    slots, x = s["slots"].long()[good], x[good]
    block, t = slots // case["bs"], slots % case["bs"]
    group = x.unflatten(2, (-1, 32))
    frac, power = torch.frexp(group.abs().amax(3))
    power = (power - torch.where(frac <= 0.875, 3, 2)).clamp(-100, 125)
    y = torch.ldexp(group, -power[..., None]).flatten(2)
    code = torch.zeros_like(y, dtype=torch.uint8)
    for k, mid in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):                     # ties go to the even code
        code += (y.abs() >= mid if k % 2 else y.abs() > mid)
    code += 8 * (y < 0)
    head = torch.arange(case["hkv"], device=DEV)[None, :, None]
    codes[block[:, None, None], head, _at4(case, t, values)[:, None]] = code[..., 0::2] + 16 * code[..., 1::2]
    scale[block[:, None, None], head, _scale_at4(case, t)[:, None]] = (power + 127).to(torch.uint8)
    out.copy_(_plain_read4(s, codes, scale, s["read"].long(), values))


def _k8_rows(x, case, back=False):
    """[.., bs * d] codes in stored order -> [.., bs, d], and back."""
    bs, d = case["bs"], case["d"]
    if back:
        return x.unflatten(-1, (d // 64, 4, 16)).unflatten(-4, (bs // 16, 16)).permute(0, 1, 2, 4, 5, 3, 6).flatten(2)
    return x.unflatten(-1, (bs // 16, d // 64, 4, 16, 16)).permute(0, 1, 2, 5, 3, 4, 6).flatten(5).flatten(4, 5).flatten(2, 3)


def _v8_rows(x, case, back=False):
    bs, d = case["bs"], case["d"]
    if back:
        return x.unflatten(-1, (d // 64, 16, 4)).unflatten(-4, (bs // 16, 4, 4)).permute(0, 1, 2, 5, 3, 6, 7, 4).flatten(2)
    return x.unflatten(-1, (bs // 16, d // 64, 4, 16, 4, 4)).permute(0, 1, 2, 4, 7, 3, 5, 6).flatten(5).flatten(2, 4)


def _values8(codes, fmt):
    return codes.view(torch.int8 if fmt == INT8 else torch.float8_e4m3fn).float()


def _plain_append8(s, x, codes, scale, order, out):
    case = s["case"]
    touched, fill, place = s["touched"], s["fill"], s["place"]
    fresh = place >= 0
    mine = x[place.clamp(min=0)].transpose(1, 2)                       # [blocks, heads, bs, d]
    fresh = fresh[:, None, :, None]
    amax = torch.where(fresh, mine.abs(), 0).amax((2, 3))
    if case["fmt"] == INT8:
        wish = amax * torch.full_like(amax, 1 / 127)
    else:
        frac, power = torch.frexp(amax)
        power = (power - torch.where(frac <= 0.875, 9, 8)).clamp(min=-126)
        wish = torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), power), 0)
    old = torch.where(fill[:, None] > 0, scale[touched], 0)
    now = torch.maximum(old, wish)
    safe = torch.where(now > 0, now, 1)
    ratio = (old / safe)[..., None, None]
    was = _values8(order(codes[touched], case), case["fmt"])
    mine = mine / safe[..., None, None]
    if case["fmt"] == INT8:
        kept, added = torch.round(was * ratio).to(torch.int8), torch.round(mine).clamp(-127, 127).to(torch.int8)
    else:
        kept, added = (was * ratio).to(torch.float8_e4m3fn), mine.clamp(-448, 448).to(torch.float8_e4m3fn)
    kept = torch.where((now > old)[..., None, None], kept.view(torch.uint8), order(codes[touched], case))
    both = torch.where(fresh, added.view(torch.uint8), kept)
    codes[touched] = order(both, case, back=True)
    scale[touched] = now
    held = (_values8(both, case["fmt"]) * now[..., None, None]).transpose(1, 2).flatten(0, 1)
    out.copy_(held[s["read_at"]])


def _rows4(codes, scale, case, values):
    """Values [blocks, heads, bs, d] of stored codes and exponents."""
    bs, D = case["bs"], case["d"]
    tiles = codes.unflatten(-1, (bs // 16, 8 * D))
    if not values:
        pair = tiles.unflatten(-1, (D // 32, 16, 16)).transpose(-3, -2).flatten(-2)          # [.., tile, t, d / 2]
    else:
        whole = D // 128 * 1024
        pair = tiles[..., :whole].unflatten(-1, (D // 128, 4, 16, 4, 4)).permute(0, 1, 2, 4, 6, 3, 5, 7).flatten(5).flatten(3, 4)
        if D % 128:
            rest = tiles[..., whole:].unflatten(-1, (4, 16, 4, 2)).permute(0, 1, 2, 3, 5, 4, 6).flatten(5).flatten(3, 4)
            pair = torch.cat([pair, rest], -1)
    pair = pair.flatten(2, 3).int()
    x = _code_values()[torch.stack([pair & 15, pair >> 4], -1)].flatten(-2)                 # [.., bs, D]
    power = scale.unflatten(-1, (bs // 16, D // 32, 16)).transpose(-2, -1).flatten(2, 3).float() - 127
    return x.unflatten(-1, (D // 32, 32)).mul_(torch.exp2(power)[..., None]).flatten(-2)


def _plain_attn(s):
    case = s["case"]
    n, hq, hkv, bs = case["n"], case["hq"], case["hkv"], case["bs"]
    group, T, most = hq // hkv, s["q"].shape[0], s["max_new"]
    start, lens, table = s["seq_start"].long(), s["lens"].long(), s["table"].long()
    token = torch.arange(T, device=DEV)
    seq = torch.searchsorted(start, token, right=True) - 1
    inside = seq < n
    seq = seq.clamp(max=n - 1)
    step = torch.where(inside, token - start[seq], most)
    q = s["q"].new_zeros((n, most + 1, hq, case["d"]), dtype=torch.float32)
    q[seq, step] = s["q"].float()
    q = q[:, :most].unflatten(2, (hkv, group)).permute(0, 2, 1, 3, 4).flatten(2, 3)          # [n, hkv, most * group, d]
    width = table.shape[1]
    safe = table.clamp(min=0).flatten()
    key = _rows4(s["k_codes"][safe], s["k_scale"][safe], case, False).unflatten(0, (n, width)).transpose(1, 2).flatten(2, 3)
    u = (q @ key.transpose(2, 3)).mul_(s["scale"])                                          # key [n, hkv, width * bs, d]
    del key
    if case["softcap"]:
        u.div_(case["softcap"]).tanh_().mul_(case["softcap"])
    at = (lens - (start[1:] - start[:-1]))[:, None] + torch.arange(most, device=DEV)        # position of each query
    at = at.repeat_interleave(group, 1)[..., None]
    j = torch.arange(width * bs, device=DEV)
    if case["alibi"]:
        slope = s["slopes"].view(1, hkv, 1, group).expand(1, hkv, most, group).flatten(2)[..., None]
        u += slope * (j - at)[:, None].float()
    seen = (j <= at) & (at < lens[:, None, None])
    if case["window"]:
        seen &= at - j < case["window"]
    u.masked_fill_(~seen[:, None], -torch.inf)
    top = u.amax(-1, keepdim=True)
    top = torch.where(top > -torch.inf, top, 0)
    u.sub_(top).exp_()
    total = u.sum(-1, keepdim=True)
    val = _rows4(s["v_codes"][safe], s["v_scale"][safe], case, True).unflatten(0, (n, width)).transpose(1, 2).flatten(2, 3)
    val.masked_fill_((j[None] >= lens[:, None])[:, None, :, None], 0)
    o = (u @ val) / torch.where(total > 0, total, 1)
    lse = torch.log(total) + top
    o = o.unflatten(2, (most, group)).permute(0, 2, 1, 3, 4).flatten(2, 3)                   # [n, most, hq, d]
    lse = lse[..., 0].unflatten(2, (most, group)).permute(0, 2, 1, 3).flatten(2, 3)
    step = step.clamp(max=most - 1)
    s["out"].copy_(torch.where(inside[:, None, None], o[seq, step].to(torch.bfloat16), s["out"]))
    s["lse"].copy_(torch.where(inside[:, None], lse[seq, step], s["lse"]))


# ------------------------------------------------------------------ the work of one pass

def work(case):
    row = case["hkv"] * case["d"]
    mx = case["fmt"] == MXFP4
    cached = row // 2 + row // 32 if mx else row                       # bytes of a token's keys or values
    scale = 0 if mx else 4 * case["hkv"]                               # and of a block's scales
    if case["op"] == "gather":
        return {"bytes": case["n"] * (2 * cached + 2 * row * (4 if case["wide"] else 2) + 4), "flops": 2 * case["n"] * row}
    before, new = _lengths(case)
    if case["op"] == "append":
        # new tokens read once and written once as codes, their queries turned; what the touched blocks hold is read back, in fp32
        some = new > 0
        first = before[some] // case["bs"]
        live = int(((before + new)[some] - first * case["bs"]).sum())
        blocks = int((-(-(before + new)[some] // case["bs"]) - first).sum())
        T, size = int(new.sum()), 4 if case["wide"] else 2
        q = T * case["hq"] * case["d"]
        return {"bytes": 2 * T * (row * size + cached) + 2 * live * (cached + 4 * row) + 4 * blocks * scale + q * (size + 2) + T * (4 * case["rot"] + 8) + 4 * live,
                "flops": 2 * row * (3 * T + live) + 3 * q}
    lens = before + new
    far = np.minimum(lens, case["window"] + new - 1) if case["window"] else lens
    pairs = sum(_pairs(int(a), int(b), case["window"]) for a, b in zip(lens, new))
    rows = int(new.sum()) * case["hq"]
    return {"bytes": int(2 * cached * far.sum() + 4 * (-(-far // case["bs"])).sum() + rows * (4 * case["d"] + 4)),
            "flops": 4 * case["d"] * case["hq"] * pairs}


def _pairs(length, new, window):
    at = np.arange(length - new, length)
    return int(np.minimum(at + 1, window).sum()) if window else int((at + 1).sum())


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "gather": _exact_gather, "attn": _exact_attn}[case["op"]](s)


def _value64(code):
    """Values of e2m1 codes from their bits."""
    e, m = code >> 1 & 3, (code & 1).double()
    mag = torch.where(e > 0, (2 + m) * torch.exp2((e - 2).double()), m / 2)
    return torch.where(code > 7, -mag, mag)


def _read64(case, codes, scale, block, t, values):
    """Cached values [tokens, d] in 64 bits; codes and scale [blocks, bytes] of one head."""
    D, d = case["d"], torch.arange(case["d"], device=DEV)
    tile, t = t // 16, (t % 16)[:, None]
    if not values:
        at = d // 32 * 256 + t * 16 + d % 32 // 2
    else:
        at = torch.where(d < D // 128 * 128, d // 128 * 1024 + t // 4 * 256 + d % 128 // 8 * 16 + t % 4 * 4 + d % 8 // 2,
                         d // 128 * 1024 + t // 4 * 128 + d % 64 // 4 * 8 + t % 4 * 2 + d % 4 // 2)
    byte = codes[block[:, None], tile[:, None] * (8 * D) + at].long()
    power = scale[block[:, None], tile[:, None] * (D // 2) + d // 32 * 16 + t].double() - 127
    return _value64(torch.where(d % 2 == 0, byte & 15, byte >> 4)) * torch.exp2(power)


def _exact_gather(s):
    case, slots = s["case"], s["slots"].long()
    got = {}
    for name in ("k", "v"):
        got[name] = torch.stack([_read64(case, s[name + "_codes"][:, h], s[name + "_scale"][:, h], slots // case["bs"], slots % case["bs"], name == "v")
                                 for h in range(case["hkv"])], 1)
    return got


def _turn64(s, x):
    """Turned channels in 64 bits; the definition rounds each product and sum to fp32."""
    if not s["case"]["rot"]:
        return x
    rot = s["case"]["rot"]
    j = torch.arange(rot, device=DEV)
    if s["case"]["pairs"]:
        angle, other, sign = j // 2, j ^ 1, torch.where(j % 2 == 0, -1.0, 1.0)
    else:
        angle, other, sign = j % (rot // 2), (j + rot // 2) % rot, torch.where(j < rot // 2, -1.0, 1.0)
    row = s["rope"].double()[s["positions"].long().clamp(0, s["rope"].shape[0] - 1)][:, None]
    cos, sin = row[..., angle], row[..., rot // 2 + angle]
    out = x.clone()
    out[..., :rot] = ((x[..., :rot] * cos).float().double() + sign * (x[..., other] * sin).float().double()).float().double()
    return out


def _round64(x, fmt):
    """The nearest value with a code, ties to even; beyond the largest, that one."""
    if fmt == INT8:
        return x.round().clamp(-127, 127)
    if fmt == MXFP4:
        step = torch.exp2((torch.frexp(x)[1] - 2).clamp(min=-1).double())
        return ((x / step).round() * step).clamp(-6, 6)
    step = torch.exp2((torch.frexp(x)[1] - 4).clamp(min=-9).double())
    return (x / step).round() * step


def _decode64(codes, fmt):
    """Values of 8-bit codes from their bits."""
    c = codes.to(torch.int64)
    if fmt == INT8:
        return torch.where(c > 127, c - 256, c).double()
    e, m = c >> 3 & 15, (c & 7).double()
    mag = torch.where(e > 0, (8 + m) * torch.exp2((e - 10).double()), m * 2.0 ** -9)
    return torch.where(c > 127, -mag, mag)


def _k8_at(case, t):
    c = torch.arange(case["d"], device=DEV)
    t = t[:, None]
    return t // 16 * (16 * case["d"]) + c // 64 * 1024 + c // 16 % 4 * 256 + t % 16 * 16 + c % 16


def _v8_at(case, t):
    c = torch.arange(case["d"], device=DEV)
    t = t[:, None]
    return t // 16 * (16 * case["d"]) + c // 64 * 1024 + t % 16 // 4 * 256 + c // 4 % 16 * 16 + c % 4 * 4 + t % 4


def _exact_append(s):
    case = s["case"]
    fmt, bs, hkv = case["fmt"], case["bs"], case["hkv"]
    read = s["read"].long()
    block, t = read // bs, read % bs
    valid = s["slots"] >= 0
    n_blocks = s["k_codes"].shape[0]
    source = torch.full((n_blocks * bs,), -1, dtype=torch.int64, device=DEV)
    source[s["slots"][valid].long()] = torch.arange(len(valid), device=DEV)[valid]
    source = source[read]
    got = {}
    for name, offsets in (("k", _k8_at), ("v", _v8_at)):
        x, codes, scale = s[name].double(), s[name + "_codes"], s[name + "_scale"]
        if name == "k":
            x = _turn64(s, x)
        if fmt == MXFP4:
            top = x.unflatten(2, (-1, 32)).abs().amax(3).clamp(min=1e-300)
            power = torch.ceil(torch.log2(top / 7)).clamp(-100, 125)
            power = torch.where(7 * torch.exp2(power) < top, power + 1, power).clamp(-100, 125)
            unit = torch.exp2(power).repeat_interleave(32, 2)
            new = _round64(x / unit, fmt) * unit
            was = torch.stack([_read64(case, codes[:, h], scale[:, h], block, t, name == "v") for h in range(hkv)], 1)
            got[name + "_out"] = torch.where((source >= 0)[:, None, None], new[source.clamp(min=0)], was)
            continue
        scale = scale.double()
        # the largest new magnitude of each (block, head), and where its live part ends
        amax = torch.zeros((n_blocks + 1, hkv), dtype=torch.float64, device=DEV)
        amax.index_reduce_(0, torch.where(valid, s["slots"].long() // bs, n_blocks), x.abs().amax(2), "amax")
        amax = amax[:-1]
        if fmt == INT8:
            wish = (amax * float(np.float32(1 / 127))).float().double()
        else:
            wish = torch.where(amax > 0, torch.exp2(torch.ceil(torch.log2((amax / 448).clamp(min=2.0 ** -126)))), 0)
        old = torch.zeros_like(scale)
        partly = s["touched"][s["fill"] > 0]
        old[partly] = scale[partly]
        now = torch.maximum(old, wish)
        ratio = (old / now.clamp(min=1e-300)).float().double()
        at = offsets(case, t)[:, None].expand(-1, hkv, -1)
        value = _decode64(codes[block].gather(2, at), fmt)
        grown = (now > old)[block][..., None]
        value = torch.where(grown, _round64((value * ratio[block][..., None]).float().double(), fmt), value)
        new = _round64((x[source.clamp(min=0)] / now[block].clamp(min=1e-300)[..., None]).float().double(), fmt)
        got[name + "_out"] = torch.where((source >= 0)[:, None, None], new, value) * now[block][..., None]
    if case["hq"]:
        known = (s["positions"] >= 0) & (s["positions"] < s["rope"].shape[0])
        got["q_out"] = torch.where(known[:, None, None], _turn64(s, s["q"].double()), s["q_out"].double())
    return got


def _exact_attn(s):
    case = s["case"]
    bs, group = case["bs"], case["hq"] // case["hkv"]
    out, lse = s["out"].double(), s["lse"].double()
    starts, lens = s["seq_start"].tolist(), s["lens"].tolist()
    for i, length in enumerate(lens):
        a, b = starts[i], starts[i + 1]
        pos = torch.arange(length, device=DEV)
        block = s["table"][i].long()[pos // bs]
        place = torch.arange(length - (b - a), length, device=DEV)
        for h in range(case["hkv"]):
            key = _read64(case, s["k_codes"][:, h], s["k_scale"][:, h], block, pos % bs, False)
            val = _read64(case, s["v_codes"][:, h], s["v_scale"][:, h], block, pos % bs, True)
            heads = torch.arange(h * group, (h + 1) * group, device=DEV)
            u = (s["q"][a:b, heads].double().flatten(0, 1) @ key.T).unflatten(0, (b - a, group)) * s["scale"]
            if case["softcap"]:
                u = case["softcap"] * torch.tanh(u / case["softcap"])
            if case["alibi"]:
                u = u + s["slopes"][heads].double()[None, :, None] * (pos - place[:, None])[:, None]
            hidden = pos > place[:, None]
            if case["window"]:
                hidden = hidden | (place[:, None] - pos >= case["window"])
            u = u.masked_fill(hidden[:, None], -torch.inf)
            lse[a:b, heads] = torch.logsumexp(u, 2)
            out[a:b, heads] = (torch.softmax(u, 2).flatten(0, 1) @ val).unflatten(0, (b - a, group))
    return {"out": out, "lse": lse}
