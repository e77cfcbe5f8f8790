"""Measured cases of the KV-cache operators: block tables and slot maps, the append into an 8-bit paged cache, its
read-back, and attention over it.

The cache holds 8-bit codes with one fp32 scale for each (block of tokens, KV head).  Codes are stored in tiles of
16 tokens, in the order a wave's matrix operands want them; for a token t of a tile and a channel d
    K: byte  (d / 64) * 1024 + (d / 16 % 4) * 256 + t * 16 + d % 16
    V: byte  (d / 64) * 1024 + (t / 4) * 256 + (d / 4 % 16) * 16 + d % 4 * 4 + t % 4
`own` false computes every operator in elementary torch operations in 32 bits, `own` true calls the library.
"""
import numpy as np
import torch

own = False

INT8, E4M3 = "int8", "e4m3"
DEV = "cuda"
GOLDEN = 0.6180339887498949


def listed():
    return [
        # the bookkeeping of one decode step of a busy server, the smallest call of a step
        dict(name="slots decode 32", op="slots", n=32, lo=1, hi=4000, prompts=0, prompt_hi=1, releases=0, bs=16, pad=0),
        # an admission step: most requests decode, some bring long prompts, some end and return their blocks
        dict(name="slots admit 250", op="slots", n=250, lo=1, hi=4000, prompts=30, prompt_hi=4000, releases=25, bs=16, pad=77),
        # one token of one request enters one layer's cache
        dict(name="append 1x1 e4m3", op="append", n=1, new_lo=1, new_hi=1, lo=100, hi=100, hkv=8, d=128, bs=16, fmt=E4M3, wide=False, pad=0),
        # a verify step: up to 9 speculated tokens of 48 requests, fp32 projections, ragged, rows of padding behind
        dict(name="append 48x9 int8", op="append", n=48, new_lo=0, new_hi=9, lo=0, hi=5000, hkv=8, d=128, bs=32, fmt=INT8, wide=True, pad=16),
        # prompts written whole
        dict(name="append prompts int8", op="append", n=13, new_lo=500, new_hi=2100, lo=0, hi=40, hkv=8, d=128, bs=64, fmt=INT8, wide=False, pad=0),
        # a shared prefix read back for a dense prompt pass
        dict(name="gather 777 e4m3", op="gather", n=777, hkv=8, d=128, bs=16, fmt=E4M3, wide=False),
        # a whole long request read back, in fp32
        dict(name="gather 32768 int8", op="gather", n=32768, hkv=8, d=128, bs=64, fmt=INT8, wide=True),
        # one request, one token: latency
        dict(name="attn 1x2048 int8", op="attn", n=1, new_lo=1, new_hi=1, lo=2048, hi=2048, hq=32, hkv=8, d=128, bs=16, fmt=INT8, softcap=0.0, window=0, alibi=False, pad=0),
        # a batch in flight, lengths from one token to 8192, one token each
        dict(name="attn 32x8192 e4m3", op="attn", n=32, new_lo=1, new_hi=1, lo=1, hi=8192, hq=32, hkv=8, d=128, bs=32, fmt=E4M3, softcap=0.0, window=0, alibi=False, pad=3),
        # a verify step of 5 tokens a request, one KV head a query head, sliding window and capped scores
        dict(name="attn verify 8x5 int8", op="attn", n=8, new_lo=5, new_hi=5, lo=300, hi=4001, hq=16, hkv=16, d=64, bs=16, fmt=INT8, softcap=30.0, window=1024, alibi=False, pad=0),
        # slices of prompts behind cached prefixes
        dict(name="attn prompts 4x300 e4m3", op="attn", n=4, new_lo=90, new_hi=300, lo=400, hi=2500, hq=32, hkv=8, d=128, bs=64, fmt=E4M3, softcap=0.0, window=0, alibi=False, pad=0),
        # long contexts, 16 query heads a KV head
        dict(name="attn 32x32768 int8", op="attn", n=32, new_lo=1, new_hi=1, lo=32768, hi=32768, hq=64, hkv=4, d=128, bs=64, fmt=INT8, softcap=0.0, window=0, alibi=False, pad=0),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["slots", "append", "gather", "attn", "attn"])
    fmt, bs, d = rng.choice([INT8, E4M3]), rng.choice([16, 32, 64, 128]), rng.choice([64, 128, 192, 256])
    if op == "slots":
        n = _log(rng, 1, 250)
        prompts = rng.randint(0, n // 8)
        return dict(op=op, n=n, lo=rng.randint(0, 50), hi=_log(rng, 60, 6000), prompts=prompts, prompt_hi=_log(rng, 1, 4000),
                    releases=rng.randint(0, (n - prompts) // 4), bs=bs, pad=rng.randint(0, 90))
    if op == "append":
        n, hkv = _log(rng, 1, 60), rng.randint(1, 12)
        hi = _log(rng, 1, max(1, 13000 // n * 8 * 128 // (hkv * d)))
        return dict(op=op, n=n, new_lo=min(hi, rng.randint(0, 2)), new_hi=hi, lo=0, hi=_log(rng, 1, 4000), hkv=hkv, d=d, bs=bs, fmt=fmt,
                    wide=rng.random() < 0.5, pad=rng.randint(0, 20))
    if op == "gather":
        hkv = rng.randint(1, 12)
        return dict(op=op, n=_log(rng, 1, max(1, 32768 * 8 * 128 // (hkv * d))), hkv=hkv, d=d, bs=bs, fmt=fmt, wide=rng.random() < 0.5)
    hkv, group = rng.randint(1, 10), rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
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
                hkv=hkv, d=d, bs=bs, fmt=fmt, softcap=softcap, window=window, alibi=alibi, pad=rng.randint(0, 5))


# ------------------------------------------------------------------ inputs

def _spread(n, lo, hi, turn):
    """n whole numbers from hi down to lo, spread evenly: the same set for every seed."""
    return hi - np.floor((np.arange(n) * turn) % 1.0 * (hi - lo + 1)).astype(np.int64)


def _lengths(case):
    """(cached before, new) tokens of each request, before the seed orders them."""
    n = case["n"]
    if case["op"] == "slots":
        new = np.ones(n, np.int64)
        new[:case["prompts"]] = _spread(case["prompts"], 1, case["prompt_hi"], GOLDEN)
        before = _spread(n, case["lo"], case["hi"], GOLDEN)
        before[:case["prompts"]] = 0
        new[n - case["releases"]:] = -1
        return before, new
    new = _spread(n, case["new_lo"], case["new_hi"], 0.7548776662466927)
    if case["op"] == "append":
        return _spread(n, case["lo"], case["hi"], GOLDEN), new
    return np.maximum(_spread(n, case["lo"], case["hi"], GOLDEN) - new, 0), new


def _cuda(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).to(DEV)


def _paged(rng, blocks, spare):
    """Block tables of requests that hold `blocks` blocks each, from a shuffled pool; (table, blocks in the pool)."""
    total = int(blocks.sum()) + spare
    pool = rng.permutation(total)
    table = np.full((len(blocks), max(1, int(blocks.max()))), -1, np.int64)
    table[np.arange(table.shape[1])[None] < blocks[:, None]] = pool[:int(blocks.sum())]
    return table, total, pool


def _codes(gen, n_blocks, hkv, width, fmt):
    out = torch.empty((n_blocks, hkv, width), dtype=torch.uint8, device=DEV)
    part = max(1, (1 << 27) // (hkv * width))
    for i in range(0, n_blocks, part):
        x = torch.randn((min(part, n_blocks - i), hkv, width), generator=gen, device=DEV)
        if fmt == INT8:
            out[i:i + part] = (x * 36).round_().clamp_(-127, 127).to(torch.int8).view(torch.uint8)
        else:
            out[i:i + part] = (x * 100).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return out


def _scales(gen, n_blocks, hkv, fmt):
    u = torch.rand((n_blocks, hkv), generator=gen, device=DEV)
    if fmt == INT8:
        return (2.6 + 1.4 * u) / 127
    return torch.where(u < 0.5, 2.0 ** -7, 2.0 ** -6)


def _cache(case, gen, n_blocks):
    width = case["bs"] * case["d"]
    s = dict(k_codes=_codes(gen, n_blocks, case["hkv"], width, case["fmt"]), v_codes=_codes(gen, n_blocks, case["hkv"], width, case["fmt"]),
             k_scale=_scales(gen, n_blocks, case["hkv"], case["fmt"]), v_scale=_scales(gen, n_blocks, case["hkv"], case["fmt"]))
    if own:
        import memory_bound_decode_amd as mbd
        fmt = mbd.MBD_KV_INT8 if case["fmt"] == INT8 else mbd.MBD_KV_E4M3
        s["cache"] = mbd.KvCache(fmt, case["bs"], case["d"], s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"])
    return s


def prepare(case, seed):
    rng = np.random.RandomState(seed % (1 << 32))
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return {"slots": _prepare_slots, "append": _prepare_append, "gather": _prepare_gather, "attn": _prepare_attn}[case["op"]](case, rng, gen)


def _prepare_slots(case, rng, gen):
    bs = case["bs"]
    before, new = _lengths(case)
    order = rng.permutation(case["n"])
    before, new = before[order], new[order]
    held = -(-before // bs)
    want = -(-(before + np.maximum(new, 0)) // bs)
    spare = int(np.maximum(want - held, 0).sum()) + 50
    table, total, pool = _paged(rng, held, spare)
    width = max(int(want.max()), table.shape[1]) + 3
    table = np.pad(table, ((0, 0), (0, width - table.shape[1])), constant_values=-1)
    free = np.full(total, -1)
    free[:spare] = pool[total - spare:]
    T = int(np.maximum(new, 0).sum()) + case["pad"]
    n = case["n"]
    s = dict(case=case, new=_cuda(new), lens=_cuda(before), held=_cuda(held), table=_cuda(table), free=_cuda(free), n_free=_cuda([spare]), T=T)
    for name, size in dict(seq_start=n + 1, slots=T, positions=T, lens_out=n, held_out=n, n_free_out=1, status=n).items():
        s[name] = torch.zeros(size, dtype=torch.int32, device=DEV)
    if own:
        import memory_bound_decode_amd as mbd
        s["pool"] = mbd.KvPool(bs, s["table"], s["free"])
    return s


def _prepare_append(case, rng, gen):
    bs, hkv, d = case["bs"], case["hkv"], case["d"]
    before, new = _lengths(case)
    order = rng.permutation(case["n"])
    before, new = before[order], new[order]
    blocks = -(-(before + new) // bs)
    table, total, _ = _paged(rng, blocks, 7)
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
    qkv = torch.randn((T, 2 * hkv * d + 64), generator=gen, device=DEV).to(dt)   # one projection's output holds both
    s = dict(case=case, k=qkv[:, :hkv * d].unflatten(1, (hkv, d)), v=qkv[:, hkv * d:2 * hkv * d].unflatten(1, (hkv, d)), slots=_cuda(slots),
             read=_cuda(read), touched=_cuda(touched, torch.int64), fill=_cuda(fill, torch.int64), place=_cuda(place, torch.int64),
             live=_cuda(all_live, torch.bool), read_at=_cuda(np.flatnonzero(all_live), torch.int64),
             k_out=torch.zeros((len(read), hkv, d), device=DEV), v_out=torch.zeros((len(read), hkv, d), device=DEV))
    return s | _cache(case, gen, total)


def _prepare_gather(case, rng, gen):
    bs = case["bs"]
    blocks = np.array([-(-case["n"] // bs)])
    table, total, _ = _paged(rng, blocks, 9)
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
    table, total, _ = _paged(rng, -(-lens // bs), 5)
    start = np.concatenate([[0], np.cumsum(new)])
    T = int(start[-1]) + case["pad"]
    s = dict(case=case, q=(torch.randn((T, hq, d), generator=gen, device=DEV) * 1.5).to(torch.bfloat16), table=_cuda(table), lens=_cuda(lens),
             seq_start=_cuda(start), out=torch.zeros((T, hq, d), dtype=torch.bfloat16, device=DEV), lse=torch.zeros((T, hq), device=DEV),
             scale=d ** -0.5, max_new=int(new.max()), max_len=int(lens.max()),
             slopes=torch.exp2(-8.0 * torch.arange(1, hq + 1, device=DEV) / hq) if case["alibi"] else None)
    s |= _cache(case, gen, total)
    if own:
        import memory_bound_decode_amd as mbd
        size = mbd.mbd_kv_attn_workspace_bytes(s["cache"], hq, n, s["max_new"], table.shape[1])
        s["ws"] = torch.zeros(size, dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    return {"slots": _run_slots, "append": _run_append, "gather": _run_gather, "attn": _run_attn}[state["case"]["op"]](state)


def _run_slots(s):
    if own:
        import memory_bound_decode_amd as mbd
        mbd.mbd_kv_slots(s["pool"], s["new"], s["lens"], s["held"], s["n_free"], s["seq_start"], s["slots"], s["positions"], s["lens_out"],
                         s["held_out"], s["n_free_out"], s["status"])
    else:
        _plain_slots(s)
    return {k: s[k] for k in ("table", "free", "seq_start", "slots", "positions", "lens_out", "held_out", "n_free_out", "status")}


def _run_append(s):
    if own:
        import memory_bound_decode_amd as mbd
        mbd.mbd_kv_append(s["cache"], s["k"], s["v"], s["slots"])
        mbd.mbd_kv_gather(s["cache"], s["read"], s["k_out"], s["v_out"])
    else:
        for x, codes, scale, order, out in (("k", "k_codes", "k_scale", _k_rows, "k_out"), ("v", "v_codes", "v_scale", _v_rows, "v_out")):
            _plain_append(s, s[x], s[codes], s[scale], order, s[out])
    return {k: s[k] for k in ("k_out", "v_out", "k_scale", "v_scale")}


def _run_gather(s):
    if own:
        import memory_bound_decode_amd as mbd
        mbd.mbd_kv_gather(s["cache"], s["slots"], s["k_out"], s["v_out"])
    else:
        bs = s["case"]["bs"]
        block, at = s["slots"].long() // bs, s["slots"].long() % bs
        s["k_out"].copy_(_token_values(s, s["k_codes"], _k_at(s["case"], at), block) * s["k_scale"][block][..., None])
        s["v_out"].copy_(_token_values(s, s["v_codes"], _v_at(s["case"], at), block) * s["v_scale"][block][..., None])
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

def _plain_slots(s):
    bs, T, width = s["case"]["bs"], s["T"], s["table"].shape[1]
    new, lens, held = s["new"].long(), s["lens"].long(), s["held"].long()
    gone, add = new < 0, new.clamp(min=0)
    start = torch.cat([add.new_zeros(1), add.cumsum(0)])
    status = torch.zeros_like(new)
    want = (lens + add + bs - 1) // bs
    status = torch.where((start[1:] > T) & (add > 0), 3, status)
    status = torch.where((want > width) & (add > 0), 2, status)
    need = torch.where((status == 0) & ~gone, (want - held).clamp(min=0), 0)
    # blocks that come back go on top of the free stack, in request order
    back = torch.where(gone, held, 0)
    col = torch.arange(width, device=DEV)[None]
    n_free = s["n_free"].long()
    spill = s["free"].shape[0]
    goes = torch.where(col < back[:, None], n_free + (back.cumsum(0) - back)[:, None] + col, spill)
    free = torch.cat([s["free"], s["free"].new_zeros(1)])
    free[goes.clamp(max=spill)] = torch.where(col < back[:, None], s["table"], 0)
    s["free"].copy_(free[:spill])
    top = n_free + back.sum()
    ends = need.cumsum(0)
    short = (need > 0) & (ends > top)
    status = torch.where(short, 1, status)
    taken = torch.where(short, 0, need)
    first = ends - need
    mine = (col >= held[:, None]) & (col < (held + taken)[:, None])
    at = (top - 1 - (first[:, None] + col - held[:, None])).clamp(0, spill - 1)
    s["table"].copy_(torch.where(mine, s["free"][at], s["table"]))
    served = (status == 0) & ~gone
    token = torch.arange(T, device=DEV)
    seq = torch.searchsorted(start, token, right=True) - 1
    inside = seq < len(new)
    seq = seq.clamp(max=len(new) - 1)
    pos = lens[seq] + token - start[seq]
    good = inside & served[seq]
    slot = s["table"][seq, (pos // bs).clamp(0, width - 1)].long() * bs + pos % bs
    s["slots"].copy_(torch.where(good, slot, -1))
    s["positions"].copy_(torch.where(good, pos, -1))
    s["seq_start"].copy_(start.clamp(max=T))
    s["lens_out"].copy_(torch.where(gone, 0, torch.where(served, lens + add, lens)))
    s["held_out"].copy_(torch.where(gone, 0, held + taken))
    s["n_free_out"].copy_(top - taken.sum())
    s["status"].copy_(status)


def _k_rows(x, case, back=False):
    """[.., bs * d] codes in stored order -> [.., bs, d], and back."""
    bs, d = case["bs"], case["d"]
    if back:
        return x.unflatten(-1, (d // 64, 4, 16)).unflatten(-4, (bs // 16, 16)).permute(0, 1, 2, 4, 5, 3, 6).flatten(2)
    return x.unflatten(-1, (bs // 16, d // 64, 4, 16, 16)).permute(0, 1, 2, 5, 3, 4, 6).flatten(5).flatten(4, 5).flatten(2, 3)


def _v_rows(x, case, back=False):
    bs, d = case["bs"], case["d"]
    if back:
        return x.unflatten(-1, (d // 64, 16, 4)).unflatten(-4, (bs // 16, 4, 4)).permute(0, 1, 2, 5, 3, 6, 7, 4).flatten(2)
    return x.unflatten(-1, (bs // 16, d // 64, 4, 16, 4, 4)).permute(0, 1, 2, 4, 7, 3, 5, 6).flatten(5).flatten(2, 4)


def _k_at(case, t):
    """Byte offsets [tokens, d] of tokens t of a block."""
    c = torch.arange(case["d"], device=DEV)
    t = t[:, None]
    return t // 16 * (16 * case["d"]) + c // 64 * 1024 + c // 16 % 4 * 256 + t % 16 * 16 + c % 16


def _v_at(case, t):
    c = torch.arange(case["d"], device=DEV)
    t = t[:, None]
    return t // 16 * (16 * case["d"]) + c // 64 * 1024 + t % 16 // 4 * 256 + c // 4 % 16 * 16 + c % 4 * 4 + t % 4


def _values(codes, fmt):
    return codes.view(torch.int8 if fmt == INT8 else torch.float8_e4m3fn).float()


def _token_values(s, codes, at, block):
    head = torch.arange(codes.shape[1], device=DEV)
    return _values(codes[block[:, None, None], head[None, :, None], at[:, None, :]], s["case"]["fmt"])


def _plain_append(s, x, codes, scale, order, out):
    case = s["case"]
    x, touched, fill, place = x.float(), s["touched"], s["fill"], s["place"]
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
    was = _values(order(codes[touched], case), case["fmt"])
    mine = mine / safe[..., None, None]
    if case["fmt"] == INT8:
        kept, added = torch.round(was * ratio).to(torch.int8), torch.round(mine).clamp(-127, 127).to(torch.int8)
    else:
        kept, added = (was * ratio).to(torch.float8_e4m3fn), mine.clamp(-448, 448).to(torch.float8_e4m3fn)
    kept = torch.where((now > old)[..., None, None], kept.view(torch.uint8), order(codes[touched], case))
    both = torch.where(fresh, added.view(torch.uint8), kept)
    codes[touched] = order(both, case, back=True)
    scale[touched] = now
    held = (_values(both, case["fmt"]) * now[..., None, None]).transpose(1, 2).flatten(0, 1)
    out.copy_(held[s["read_at"]])


def _plain_attn(s):
    case = s["case"]
    n, hq, hkv, d, bs, fmt = case["n"], case["hq"], case["hkv"], case["d"], case["bs"], case["fmt"]
    group, T, most = hq // hkv, s["q"].shape[0], s["max_new"]
    start, lens, table = s["seq_start"].long(), s["lens"].long(), s["table"].long()
    token = torch.arange(T, device=DEV)
    seq = torch.searchsorted(start, token, right=True) - 1
    inside = seq < n
    seq = seq.clamp(max=n - 1)
    step = torch.where(inside, token - start[seq], most)
    q = s["q"].new_zeros((n, most + 1, hq, d), dtype=torch.float32)
    q[seq, step] = s["q"].float()
    q = q[:, :most].unflatten(2, (hkv, group)).permute(0, 2, 1, 3, 4).flatten(2, 3)          # [n, hkv, most * group, d]
    width = table.shape[1]
    safe = table.clamp(min=0)
    key = _values(_k_rows(s["k_codes"][safe].flatten(0, 1), case), fmt).unflatten(0, (n, width))
    key.mul_(s["k_scale"][safe][..., None, None])
    key = key.transpose(1, 2).flatten(2, 3)                                                 # [n, hkv, width * bs, d]
    u = (q @ key.transpose(2, 3)).mul_(s["scale"])
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
    val = _values(_v_rows(s["v_codes"][safe].flatten(0, 1), case), fmt).unflatten(0, (n, width))
    val.mul_(s["v_scale"][safe][..., None, None])
    val = val.transpose(1, 2).flatten(2, 3)
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
    if case["op"] == "slots":
        before, new = _lengths(case)
        add = np.maximum(new, 0)
        fresh = np.maximum(-(-(before + add) // case["bs"]) + (-before // case["bs"]), 0).sum()
        back = np.where(new < 0, -(-before // case["bs"]), 0).sum()
        return {"bytes": int(case["n"] * 28 + 8 * (add.sum() + case["pad"]) + 8 * fresh + 8 * back), "flops": 0}
    row = case["hkv"] * case["d"]
    if case["op"] == "gather":
        return {"bytes": case["n"] * (2 * row * (1 + (4 if case["wide"] else 2)) + 4) + 8 * case["hkv"] * -(-case["n"] // case["bs"]), "flops": 2 * case["n"] * row}
    before, new = _lengths(case)
    if case["op"] == "append":
        # new tokens read once and written once as codes; what the touched blocks hold is read back, in fp32
        some = new > 0
        live = int(((before + new)[some] - before[some] // case["bs"] * case["bs"]).sum())
        T = int(new.sum())
        return {"bytes": 2 * row * (T * ((4 if case["wide"] else 2) + 1) + live * (1 + 4)) + 4 * (T + live), "flops": 2 * row * (3 * T + live)}
    lens = before + new
    far = np.minimum(lens, case["window"] + new - 1) if case["window"] else lens
    pairs = sum(_pairs(int(a), int(b), case["window"]) for a, b in zip(lens, new))
    rows = int(new.sum()) * case["hq"]
    return {"bytes": int(2 * row * far.sum() + 8 * case["hkv"] * (-(-far // case["bs"])).sum() + 4 * (-(-far // case["bs"])).sum() + rows * (4 * case["d"] + 4)),
            "flops": 4 * case["d"] * case["hq"] * pairs}


def _pairs(length, new, window):
    at = np.arange(length - new, length)
    return int(np.minimum(at + 1, window).sum()) if window else int((at + 1).sum())


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    if case["op"] == "slots":
        return None
    s = prepare(case, seed)
    return {"append": _exact_append, "gather": _exact_gather, "attn": _exact_attn}[case["op"]](s)


def _decode64(codes, fmt):
    """Values of 8-bit codes from their bits."""
    c = codes.to(torch.int64)
    if fmt == INT8:
        return torch.where(c > 127, c - 256, c).double()
    e, m = c >> 3 & 15, (c & 7).double()
    mag = torch.where(e > 0, (8 + m) * torch.exp2((e - 10).double()), m * 2.0 ** -9)
    return torch.where(c > 127, -mag, mag)


def _round64(x, fmt):
    """The nearest value with an 8-bit code, ties to even."""
    if fmt == INT8:
        return x.round().clamp(-127, 127)
    step = torch.exp2((torch.frexp(x)[1] - 4).clamp(min=-9).double())
    return (x / step).round() * step


def _exact_gather(s):
    case, slots = s["case"], s["slots"].long()
    block, t = slots // case["bs"], slots % case["bs"]
    got = {}
    for name, offsets in (("k", _k_at), ("v", _v_at)):
        codes = s[name + "_codes"][block]                                # [n, heads, bs * d]
        at = offsets(case, t)[:, None].expand(-1, case["hkv"], -1)
        got[name] = _decode64(codes.gather(2, at), case["fmt"]) * s[name + "_scale"][block].double()[..., None]
    return got


def _exact_append(s):
    case = s["case"]
    fmt, bs, hkv, d = case["fmt"], case["bs"], case["hkv"], case["d"]
    got = {}
    token_block = torch.where(s["slots"] >= 0, s["slots"].long() // bs, -1)
    for name, offsets in (("k", _k_at), ("v", _v_at)):
        x, codes, scale = s[name].double(), s[name + "_codes"], s[name + "_scale"].double()
        # the largest new magnitude of each (block, head), and where its live part ends
        amax = torch.zeros((codes.shape[0] + 1, hkv), dtype=torch.float64, device=DEV)
        amax.index_reduce_(0, token_block % (codes.shape[0] + 1), x.abs().amax(2), "amax")
        amax = amax[:-1]
        if fmt == INT8:
            wish = (amax * float(np.float32(1 / 127))).float().double()
        else:
            wish = torch.where(amax > 0, torch.exp2(torch.ceil(torch.log2((amax / 448).clamp(min=2.0 ** -126)))), 0)
        old = torch.zeros_like(scale)
        partly = s["touched"][s["fill"] > 0]
        old[partly] = scale[partly]
        hit = torch.zeros(codes.shape[0], dtype=torch.bool, device=DEV)
        hit[s["touched"]] = True
        now = torch.where(hit[:, None], torch.maximum(old, wish), scale)
        ratio = (old / now.clamp(min=1e-300)).float().double()
        read = s["read"].long()
        block, t = read // bs, read % bs
        at = offsets(case, t)[:, None].expand(-1, hkv, -1)
        value = _decode64(codes[block].gather(2, at), fmt)
        grown = (now > old)[block][..., None]
        value = torch.where(grown, _round64((value * ratio[block][..., None]).float().double(), fmt), value)
        source = torch.full((codes.shape[0] * bs,), -1, dtype=torch.int64, device=DEV)
        valid = s["slots"] >= 0
        source[s["slots"][valid].long()] = torch.arange(len(valid), device=DEV)[valid]
        source = source[read]
        new = _round64((x[source.clamp(min=0)] / now[block].clamp(min=1e-300)[..., None]).float().double(), fmt)
        got[name + "_out"] = torch.where((source >= 0)[:, None, None], new, value) * now[block][..., None]
        got[name + "_scale"] = now
    return got


def _exact_attn(s):
    case = s["case"]
    bs, hkv, group, d = case["bs"], case["hkv"], case["hq"] // case["hkv"], case["d"]
    out, lse = s["out"].double(), s["lse"].double()
    starts, lens = s["seq_start"].tolist(), s["lens"].tolist()
    for i, length in enumerate(lens):
        a, b = starts[i], starts[i + 1]
        pos = torch.arange(length, device=DEV)
        block = s["table"][i].long()[pos // bs]
        kept = {}
        for name, offsets in (("k", _k_at), ("v", _v_at)):
            blocks, back = torch.unique(block, return_inverse=True)
            at = offsets(case, pos % bs)
            for h in range(hkv):
                codes = s[name + "_codes"][blocks, h]
                kept[name, h] = _decode64(codes[back[:, None], at], case["fmt"]) * s[name + "_scale"][block, h].double()[:, None]
        place = torch.arange(length - (b - a), length, device=DEV)
        for h in range(case["hq"]):
            u = s["q"][a:b, h].double() @ kept["k", h // group].T * s["scale"]
            if case["softcap"]:
                u = case["softcap"] * torch.tanh(u / case["softcap"])
            if case["alibi"]:
                u = u + s["slopes"][h].double() * (pos[None] - place[:, None])
            hidden = pos[None] > place[:, None]
            if case["window"]:
                hidden = hidden | (place[:, None] - pos[None] >= case["window"])
            u = u.masked_fill(hidden, -torch.inf)
            lse[a:b, h] = torch.logsumexp(u, 1)
            out[a:b, h] = torch.softmax(u, 1) @ kept["v", h // group]
    return {"out": out, "lse": lse}
