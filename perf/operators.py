"""Cases of the serving-step operators beside the paged cache: block tables and
slots built on the GPU, rotary positions with the cache write, a cache held in
4 bits (append, read back, attention), and windowed attention with sinks.

Each case is one pass of one operator as a decode or prefill step calls it;
``run`` computes it in its plain form (elementary torch operations, 32 bits,
rounded once at the end) or, with ``own`` true, through the package.

The 4-bit cache, as include/pagedkv.h lays it out: a (block, KV head) tile
holds block_size / 16 sub-tiles of 16 tokens; a sub-tile is 16 rows of
head_dim / 2 code bytes (two codes a byte, the lower nibble first), then
[16][head_dim / 64] pairs (scale, minimum) in bf16, one per 64 dims of a
token. Within a row the codes are permuted (``code_places``). A value is
minimum + scale * code.
"""

import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------
# Cases

def listed():
    return [
        # a decode step's bookkeeping: one new token for each sequence of a ragged batch
        {"name": "extend_decode", "op": "extend", "B": 256, "lo": 16, "hi": 8192, "new_lo": 1,
         "new_hi": 1, "bs": 16, "release": 0, "pad": 0, "lens_seed": 1},
        # a prefill wave: prompts and chunks of very different lengths, some sequences leaving
        {"name": "extend_prefill", "op": "extend", "B": 512, "lo": 1, "hi": 4096, "new_lo": 1,
         "new_hi": 8192, "bs": 16, "release": 40, "pad": 1000, "lens_seed": 2},
        # one token of one request: latency
        {"name": "rope_token", "op": "rope", "T": 1, "Hq": 32, "Hkv": 8, "D": 128, "rd": 128,
         "bs": 16, "dtype": "bf16", "layout": "half", "scaling": "none", "factor": 1.0,
         "far": 8192, "fused": False},
        # a prefill of 16 x 1024 tokens with stretched frequencies, q, k and v as views of one product
        {"name": "rope_prefill", "op": "rope", "T": 16384, "Hq": 32, "Hkv": 8, "D": 128, "rd": 128,
         "bs": 16, "dtype": "bf16", "layout": "half", "scaling": "yarn", "factor": 16.0,
         "far": 131072, "fused": True},
        # part of the head, interleaved pairs, fp32, an odd number of tokens
        {"name": "rope_partial_f32", "op": "rope", "T": 777, "Hq": 16, "Hkv": 16, "D": 64, "rd": 32,
         "bs": 32, "dtype": "f32", "layout": "interleaved", "scaling": "linear", "factor": 4.0,
         "far": 32768, "fused": True},
        # the 4-bit cache's write in a decode step: one token for each of 256 sequences
        {"name": "append4_decode", "op": "append4", "T": 256, "Hkv": 8, "D": 128, "bs": 16},
        # and in a prefill of 16 x 1024 tokens
        {"name": "append4_prefill", "op": "append4", "T": 16384, "Hkv": 8, "D": 128, "bs": 16},
        # attention over the 4-bit cache: the smallest step (lengths 1, 15, 16, 33)
        {"name": "decode4_tiny", "op": "decode4", "B": 4, "lo": 1, "hi": 33, "Hq": 2, "Hkv": 2,
         "D": 64, "bs": 16, "window": 0, "sinks": 0, "lens": "tiny", "lens_seed": 0},
        # a ragged grouped-query batch
        {"name": "decode4_gqa", "op": "decode4", "B": 256, "lo": 16, "hi": 8192, "Hq": 32, "Hkv": 8,
         "D": 128, "bs": 16, "window": 0, "sinks": 0, "lens": "log", "lens_seed": 3},
        # long contexts
        {"name": "decode4_long", "op": "decode4", "B": 8, "lo": 131072, "hi": 131072, "Hq": 64,
         "Hkv": 8, "D": 128, "bs": 16, "window": 0, "sinks": 0, "lens": "log", "lens_seed": 4},
        # a short window with sinks over ragged lengths, fp32
        {"name": "sinks_f32", "op": "sinks", "B": 7, "lo": 1, "hi": 700, "Hq": 4, "Hkv": 2, "D": 64,
         "bs": 16, "window": 97, "sinks": 4, "dtype": "f32", "lens_seed": 5},
        # a 4096-token window with sinks at long contexts; blocks before the window are released
        {"name": "sinks_long", "op": "sinks", "B": 8, "lo": 100000, "hi": 131072, "Hq": 64, "Hkv": 8,
         "D": 128, "bs": 16, "window": 4096, "sinks": 4, "dtype": "bf16", "lens_seed": 6},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["extend", "rope", "append4", "decode4", "decode4", "sinks"])
    seed = rng.randrange(1 << 20)
    bs = rng.choice([16, 32])
    if op == "extend":
        new_hi = rng.choice([1, _log(rng, 1, 4096)])
        return {"op": op, "B": _log(rng, 1, 700), "lo": 1, "hi": _log(rng, 16, 8192), "new_lo": 1,
                "new_hi": new_hi, "bs": bs, "release": rng.choice([0, rng.randrange(100)]),
                "pad": rng.choice([0, rng.randrange(3000)]), "lens_seed": seed}
    heads, D = rng.choice([(1, 1), (2, 2), (8, 2), (32, 8), (32, 32), (12, 2), (16, 1), (64, 8)]), rng.choice([64, 128, 256])
    if op == "rope":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        return {"op": op, "T": _log(rng, 1, 4000), "Hq": heads[0], "Hkv": heads[1], "D": D,
                "rd": rng.choice([D, D, D // 2, 32, 48]), "bs": bs, "dtype": dtype,
                "layout": rng.choice(["half", "interleaved"]),
                "scaling": rng.choice(["none", "linear", "ntk", "yarn"]),
                "factor": rng.choice([2.0, 8.0, 32.0]), "far": _log(rng, 100, 1000000),
                "fused": rng.random() < 0.5}
    if op == "append4":
        return {"op": op, "T": _log(rng, 1, 8000), "Hkv": heads[1], "D": D, "bs": bs}
    B = _log(rng, 1, 200)
    hi = _log(rng, 2, min(131072, max(2, 300000000 // (B * heads[1] * D))))
    case = {"op": op, "B": B, "lo": 1 + rng.randrange(hi), "hi": hi, "Hq": heads[0], "Hkv": heads[1],
            "D": D, "bs": bs, "lens_seed": seed}
    if op == "decode4":
        windowed = rng.random() < 0.4
        return {**case, "window": _log(rng, 1, hi) if windowed else 0,
                "sinks": rng.choice([0, 1, 4, 37]) if windowed else 0, "lens": "log"}
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if dtype == "f32":
        case["Hq"], case["Hkv"], case["D"] = rng.choice([(1, 1), (8, 2), (8, 1)]) + (rng.choice([64, 128]),)
    return {**case, "dtype": dtype, "window": _log(rng, 1, min(hi, 8192)), "sinks": rng.choice([1, 4, 16, 37])}


def _dtype(case):
    return torch.float32 if case.get("dtype") == "f32" else torch.bfloat16


def _lengths(case):
    """The batch's context lengths, fixed by the case alone."""
    if case.get("lens") == "tiny":
        return [1, 15, 16, 33]
    rng = random.Random(case["lens_seed"])
    return [_log(rng, case["lo"], case["hi"]) for _ in range(case["B"])]


def _new_lengths(case):
    """New tokens of each sequence of an extend case; -1 leaves the batch."""
    rng = random.Random(case["lens_seed"] + 7)
    new = [_log(rng, case["new_lo"], case["new_hi"]) for _ in range(case["B"])]
    return [-1 if rng.randrange(1000) < case["release"] else n for n in new]


def _visible(case):
    """Tokens that each sequence's query sees."""
    W, S = case["window"], case["sinks"]
    return [c if not W else min(c, W) + min(S, max(0, c - W)) for c in _lengths(case)]


# ---------------------------------------------------------------------------
# The 4-bit tile's layout

def code_places(D, value):
    """[16, D]: where the code of (token of the sub-tile, dim) stands among the
    row's D nibbles, for K (value false) and V (value true)."""
    tok = torch.arange(16, device=DEV)[:, None]
    d = torch.arange(D, device=DEV)[None, :]
    if value:
        turn = {64: 0 * tok, 128: 4 * ((tok >> 1) & 1), 256: 2 * (tok & 3)}[D]
        return (((d >> 3) & 7) ^ turn) * (D // 8) + (d >> 6) * 8 + (d & 7)
    word = 2 * (d >> 6) + ((d >> 3) & 1)
    if D == 64:
        return (d + 0 * tok)
    panel = (word >> 2) ^ ((tok & 1) if D == 256 else 0 * tok)
    return panel * 128 + ((d >> 4) & 3) * 32 + (word & 3) * 8 + (d & 7)


def tile_bytes(bs, D):
    return bs // 16 * 9 * D


# ---------------------------------------------------------------------------
# Inputs

def _tables(case, lens, gen, slack=0, live=None):
    """Shuffled block tables (-1 past each sequence's end, and where `live`
    says that a block is released), and the number of blocks of the pool."""
    bs = case["bs"]
    mbs = max(1, max((n + bs - 1) // bs for n in lens)) + slack
    want = torch.zeros(len(lens), mbs, dtype=torch.bool)
    for s, n in enumerate(lens):
        want[s, :(n + bs - 1) // bs] = True
        if live is not None:
            want[s] &= live(s, torch.arange(mbs))
    total = int(want.sum())
    nb = max(1, total + total // 10 + 4)
    table = torch.full(want.shape, -1, dtype=torch.int32)
    order = torch.randperm(nb, generator=gen, device=DEV).cpu()
    table[want] = order[:total].to(torch.int32)
    return table.to(DEV), nb, order[total:].to(torch.int32)


def _packed_pool(nb, case, gen):
    """A 4-bit pool of random codes, scales near 0.3 and minima near -7.5 scales."""
    Hkv, D, U = case["Hkv"], case["D"], case["bs"] // 16
    pool = torch.randint(0, 256, (nb, Hkv, U, 9 * D), dtype=torch.uint8, device=DEV, generator=gen)
    s = torch.rand(nb, Hkv, U, 16, D // 64, device=DEV, generator=gen) * 0.2 + 0.2
    m = -7.5 * s + 0.2 * torch.randn(s.shape, device=DEV, generator=gen)
    pool[..., 8 * D:] = torch.stack([s, m], -1).to(torch.bfloat16).view(torch.uint8).flatten(3)
    return pool.view(nb, Hkv, U * 9 * D)


def frequencies(case):
    """Inverse frequencies (fp32) and the factor on cos and sin, base 10000:
    "linear" divides positions by the factor, "ntk" stretches the base, "yarn"
    ramps between kept (over 32 turns in the original 4096 tokens) and divided
    (under 1 turn) frequencies and scales by 0.1 ln(factor) + 1."""
    rd, f = case["rd"], case["factor"]
    i = np.arange(rd // 2, dtype=np.float64)
    base = 10000.0
    if case["scaling"] == "ntk":
        base *= f ** (rd / (rd - 2.0))
    inv = base ** (-2.0 * i / rd)
    m = 1.0
    if case["scaling"] == "linear":
        inv = inv / f
    if case["scaling"] == "yarn":
        def dim(turns):
            return rd * math.log(4096.0 / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))
        low, high = max(math.floor(dim(32.0)), 0), min(math.ceil(dim(1.0)), rd - 1)
        ramp = np.clip((i - low) / max(high - low, 0.001), 0.0, 1.0)
        inv = inv / f * ramp + inv * (1.0 - ramp)
        m = 0.1 * math.log(f) + 1.0
    return inv.astype(np.float32), m


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(1000003 * seed + 17)
    st = {"case": case, "scale": 1.0 / math.sqrt(case.get("D", 64))}
    op, dt = case["op"], _dtype(case)

    def normal(*shape, dtype=dt):
        return torch.randn(*shape, device=DEV, generator=gen).to(dtype)

    if op == "extend":
        lens, new = _lengths(case), _new_lengths(case)
        rows = [n + max(0, k) for n, k in zip(lens, new)]
        bs = case["bs"]
        held, nb, _ = _tables(case, rows, gen)
        # blocks past each sequence's present end are still in the queue
        mbs = held.shape[1]
        have = torch.tensor([(n + bs - 1) // bs for n in lens], device=DEV)
        st["tables"] = torch.where(torch.arange(mbs, device=DEV)[None] < have[:, None], held, -1).to(torch.int32)
        used = torch.zeros(nb, dtype=torch.bool, device=DEV)
        used[st["tables"][st["tables"] >= 0].long()] = True
        free = torch.nonzero(~used)[:, 0].to(torch.int32)
        free = free[torch.randperm(free.numel(), device=DEV, generator=gen)]
        head = nb // 3
        queue = torch.full((nb,), -1, dtype=torch.int32, device=DEV)
        queue[(head + torch.arange(free.numel(), device=DEV)) % nb] = free
        st["queue"] = queue
        st["queue_state"] = torch.tensor([head, free.numel()], dtype=torch.int32, device=DEV)
        st["ctx"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        st["new"] = torch.tensor(new, dtype=torch.int32, device=DEV)
        st["max_tokens"] = sum(max(0, k) for k in new) + case["pad"]
        return st
    if op == "rope":
        T, Hq, Hkv, D, bs = case["T"], case["Hq"], case["Hkv"], case["D"], case["bs"]
        if case["fused"]:
            qkv = normal(T, (Hq + 2 * Hkv) * D)
            q, k, v = qkv[:, :Hq * D], qkv[:, Hq * D:(Hq + Hkv) * D], qkv[:, (Hq + Hkv) * D:]
            st["q"], st["k"], st["v"] = q.unflatten(1, (Hq, D)), k.unflatten(1, (Hkv, D)), v.unflatten(1, (Hkv, D))
        else:
            st["q"], st["k"], st["v"] = normal(T, Hq, D), normal(T, Hkv, D), normal(T, Hkv, D)
        nb = (T + bs - 1) // bs + 4
        st["k_pool"], st["v_pool"] = normal(nb, Hkv, bs, D), normal(nb, Hkv, bs, D)
        st["slots"] = torch.randperm(nb * bs, device=DEV, generator=gen)[:T]
        start = int(torch.randint(0, max(1, case["far"] - T + 1), (1,), device=DEV, generator=gen))
        st["positions"] = torch.arange(start, start + T, dtype=torch.int32, device=DEV)
        inv, st["mscale"] = frequencies(case)
        st["inv_freq"] = torch.from_numpy(inv).to(DEV)
        return st
    if op == "append4":
        T, Hkv, D, bs = case["T"], case["Hkv"], case["D"], case["bs"]
        spread = torch.exp(0.5 * torch.randn(Hkv, D, device=DEV, generator=gen))  # channels differ in size
        st["k"] = (torch.randn(T, Hkv, D, device=DEV, generator=gen) * spread).to(dt)
        st["v"] = normal(T, Hkv, D)
        nb = (T + bs - 1) // bs + 4
        st["k_pool"], st["v_pool"] = _packed_pool(nb, case, gen), _packed_pool(nb, case, gen)
        st["slots"] = torch.randperm(nb * bs, device=DEV, generator=gen)[:T]
        return st
    lens = _lengths(case)
    B, Hq, Hkv, D, bs, W, S = (case[x] for x in ("B", "Hq", "Hkv", "D", "bs", "window", "sinks"))
    st["q"] = normal(B, Hq, D)
    st["ctx"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    if op == "decode4":
        st["tables"], nb, _ = _tables(case, lens, gen, slack=1)
        st["k_pool"], st["v_pool"] = _packed_pool(nb, case, gen), _packed_pool(nb, case, gen)
        return st

    def live(s, b):  # blocks that hold a sink or a token of the window
        return (b * bs < S) | ((b + 1) * bs > lens[s] - W)

    st["tables"], nb, _ = _tables(case, lens, gen, slack=1, live=live)
    st["k_pool"], st["v_pool"] = normal(nb, Hkv, bs, D), normal(nb, Hkv, bs, D)
    return st


# ---------------------------------------------------------------------------
# One pass

def run(st):
    op = st["case"]["op"]
    if own:
        return _own(st, op)
    return {"extend": _plain_extend, "rope": _plain_rope, "append4": _plain_append4,
            "decode4": _plain_decode4, "sinks": _plain_sinks}[op](st)


def _own(st, op):
    from paged_kv_cache_336_b200 import binding
    case = st["case"]
    if op == "extend":
        if "next" not in st:  # a serving loop keeps two sets of a step's outputs and swaps them
            st["next"] = binding.StepTables.empty(case["B"], st["max_tokens"])
        r = binding.extend_tables(st["tables"], st["ctx"], st["new"], st["queue"], st["queue_state"],
                                  case["bs"], st["max_tokens"], out=st["next"])
        return [st["tables"], r.context_lens, r.query_start, r.positions, r.slot_mapping, r.queue_state, st["queue"]]
    if op == "rope":
        q = binding.rope_append(st["q"], st["k"], st["v"], st["positions"], st["inv_freq"], st["slots"],
                                st["k_pool"], st["v_pool"], interleaved=case["layout"] == "interleaved",
                                mscale=st["mscale"])
        return [q, st["k_pool"], st["v_pool"]]
    if op == "append4":
        binding.kv_append_q4(st["k"], st["v"], st["slots"], st["k_pool"], st["v_pool"])
        return list(binding.kv_gather_q4(st["k_pool"], st["v_pool"], st["slots"], case["D"]))
    if "workspace" not in st:  # a serving loop keeps one
        st["workspace"] = binding.SplitWorkspace(case["B"], case["Hq"], case["D"], case["bs"],
                                                 st["tables"].shape[1], 512)
    if op == "decode4":
        return binding.decode_q4(st["q"], st["k_pool"], st["v_pool"], st["tables"], st["ctx"], st["scale"],
                                 window=case["window"], sinks=case["sinks"], workspace=st["workspace"])
    return binding.decode_split_sinks(st["q"], st["k_pool"], st["v_pool"], st["tables"], st["ctx"],
                                      st["scale"], case["window"], case["sinks"], workspace=st["workspace"])


def _plain_extend(st):
    bs, T = st["case"]["bs"], st["max_tokens"]
    tables, ctx, queue = st["tables"], st["ctx"].long(), st["queue"]
    new = st["new"].long().clamp(min=0)
    gone = st["new"] < 0
    have = (ctx + bs - 1) // bs
    need = (ctx + new + bs - 1) // bs - have
    back = torch.where(gone, have, 0)
    taken, given = torch.cumsum(need, 0), torch.cumsum(back, 0)
    head, count, cap = st["queue_state"][0].long(), st["queue_state"][1].long(), queue.numel()
    j = torch.arange(tables.shape[1], device=DEV)[None]
    fresh = (j >= have[:, None]) & (j < (have + need)[:, None])
    src = (head + (taken - need)[:, None] + j - have[:, None]) % cap
    tables.copy_(torch.where(fresh, queue[src], tables))
    # blocks of the leaving sequences, in order, behind the queue's end
    i = torch.arange(cap, device=DEV)
    s = torch.searchsorted(given, i, right=True).clamp(max=ctx.numel() - 1)
    block = tables[s, (i - (given - back)[s]).clamp(0, tables.shape[1] - 1)]
    at = (head + count + i) % cap
    queue[at] = torch.where(i < given[-1], block, queue[at])
    start = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), torch.cumsum(new, 0)])
    t = torch.arange(T, device=DEV)
    seq = torch.searchsorted(start[1:], t, right=True).clamp(max=ctx.numel() - 1)
    real = t < start[-1]
    pos = ctx[seq] + t - start[seq]
    slot = tables[seq, (pos // bs).clamp(max=tables.shape[1] - 1)].long() * bs + pos % bs
    after = torch.where(gone, 0, ctx + new)
    state = torch.stack([(head + taken[-1]) % cap, count - taken[-1] + given[-1]])
    return [tables, after.int(), start.int(), torch.where(real, pos, 0).int(),
            torch.where(real, slot, -1), state.int(), queue]


def _rotate(x, cos, sin, rd, layout):
    a, rest = x[..., :rd].float(), x[..., rd:].float()
    if layout == "half":
        lo, hi = a[..., :rd // 2], a[..., rd // 2:]
        a = torch.cat([lo * cos - hi * sin, hi * cos + lo * sin], -1)
    else:
        lo, hi = a[..., 0::2], a[..., 1::2]
        a = torch.stack([lo * cos - hi * sin, hi * cos + lo * sin], -1).flatten(-2)
    return torch.cat([a, rest], -1).to(x.dtype)


def _plain_rope(st):
    case = st["case"]
    # angles of far positions need more than 32 bits
    f = st["positions"].double()[:, None] * st["inv_freq"].double()[None]
    cos = (torch.cos(f) * st["mscale"]).float()[:, None]
    sin = (torch.sin(f) * st["mscale"]).float()[:, None]
    q = _rotate(st["q"], cos, sin, case["rd"], case["layout"])
    k = _rotate(st["k"], cos, sin, case["rd"], case["layout"])
    block, off = st["slots"] // case["bs"], st["slots"] % case["bs"]
    st["k_pool"][block, :, off] = k
    st["v_pool"][block, :, off] = st["v"]
    return [q, st["k_pool"], st["v_pool"]]


def _codes(x):
    """Codes, scales and minima of bf16 rows: one group per 64 dims."""
    g = x.float().unflatten(-1, (-1, 64))
    low = g.amin(-1)
    scale = ((g.amax(-1) - low) / 15.0).to(torch.bfloat16).float()
    code = torch.round((g - low[..., None]) / torch.where(scale > 0, scale, 1.0)[..., None]).clamp(0, 15)
    return torch.where(scale[..., None] > 0, code, 0).to(torch.uint8).flatten(-2), scale, low


def _write4(pool, x, slots, bs, value):
    T, Hkv, D = x.shape
    code, scale, low = _codes(x)
    tok = slots % bs
    place = code_places(D, value)[tok % 16][:, None].expand(T, Hkv, D)
    nib = torch.empty_like(code).scatter_(2, place, code)
    sub = pool.view(pool.shape[0], Hkv, bs // 16, 9 * D)
    sub[..., :8 * D].unflatten(3, (16, D // 2))[slots // bs, :, tok // 16, tok % 16] = nib[..., 0::2] | (nib[..., 1::2] << 4)
    both = torch.stack([scale, low], -1).to(torch.bfloat16).view(torch.uint8).flatten(2)
    sub[..., 8 * D:].unflatten(3, (16, D // 16))[slots // bs, :, tok // 16, tok % 16] = both


def _read4(pool, slots, D, bs, value):
    Hkv = pool.shape[1]
    tok = slots % bs
    sub = pool.view(pool.shape[0], Hkv, bs // 16, 9 * D)
    row = sub[..., :8 * D].unflatten(3, (16, D // 2))[slots // bs, :, tok // 16, tok % 16]
    both = sub[..., 8 * D:].unflatten(3, (16, D // 16))[slots // bs, :, tok // 16, tok % 16]
    both = both.contiguous().view(torch.bfloat16).float().unflatten(2, (D // 64, 2))
    nib = torch.stack([row & 15, row >> 4], -1).flatten(2)
    place = code_places(D, value)[tok % 16][:, None].expand(slots.numel(), Hkv, D)
    code = torch.gather(nib, 2, place).float().unflatten(2, (-1, 64))
    return (both[..., 1:] + both[..., :1] * code).flatten(2)


def _plain_append4(st):
    case = st["case"]
    out = []
    for name, value in (("k", False), ("v", True)):
        _write4(st[name + "_pool"], st[name], st["slots"], case["bs"], value)
        out.append(_read4(st[name + "_pool"], st["slots"], case["D"], case["bs"], value).to(torch.bfloat16))
    return out


def _expand4(tiles, bs, D, value):
    """[B, mbs, Hkv, tile bytes] -> values [B, Hkv, mbs * bs, D]."""
    B, mbs, Hkv = tiles.shape[:3]
    sub = tiles.view(B, mbs, Hkv, bs // 16, 9 * D)
    codes = sub[..., :8 * D]
    nib = torch.stack([codes & 15, codes >> 4], -1).flatten(4)
    place = (code_places(D, value) + D * torch.arange(16, device=DEV)[:, None]).flatten()
    code = nib[..., place].unflatten(4, (16, D // 64, 64))
    both = sub[..., 8 * D:].contiguous().view(torch.bfloat16).float().unflatten(4, (16, D // 64, 2))
    x = both[..., 1:] + both[..., :1] * code.float()
    return x.permute(0, 2, 1, 3, 4, 5, 6).reshape(B, Hkv, mbs * bs, D)


def _attend(q, k, v, see, scale):
    """softmax(scale q k^T) v over the tokens that `see` [B, L] marks; zeros for none."""
    B, Hq, D = q.shape
    Hkv = k.shape[1]
    x = (q.float().view(B, Hkv, Hq // Hkv, D) @ k.transpose(2, 3)) * scale
    x = x.masked_fill(~see[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(torch.isinf(top), 0.0, top))
    total = p.sum(-1, keepdim=True)
    out = (p @ v) / torch.where(total > 0, total, 1.0)
    return out.reshape(B, Hq, D).to(q.dtype)


def _plain_decode4(st):
    case, tables = st["case"], st["tables"]
    bs, D, W = case["bs"], case["D"], case["window"]
    ctx = st["ctx"].long()[:, None]
    t = torch.arange(tables.shape[1] * bs, device=DEV)[None]
    see = t < ctx
    if W:
        see = see & ((t >= ctx - W) | (t < case["sinks"]))
    at = tables.clamp(min=0).long()
    k = _expand4(st["k_pool"][at], bs, D, False)
    v = _expand4(st["v_pool"][at], bs, D, True)
    return _attend(st["q"], k, v, see, st["scale"])


def _plain_sinks(st):
    case, tables = st["case"], st["tables"]
    bs, W, S = case["bs"], case["window"], case["sinks"]
    ctx = st["ctx"].long()[:, None]
    first = torch.arange(S, device=DEV)[None].expand(ctx.shape[0], S)
    last = ctx - W + torch.arange(W, device=DEV)[None]
    t = torch.cat([first, last], 1)
    see = torch.cat([first < ctx, last >= S], 1)  # a sink inside the window counts once
    t = torch.where(see, t, 0)
    block = tables.gather(1, t // bs).clamp(min=0).long()
    k = st["k_pool"][block, :, t % bs].float().transpose(1, 2)
    v = st["v_pool"][block, :, t % bs].float().transpose(1, 2)
    return _attend(st["q"], k, v, see, st["scale"])


# ---------------------------------------------------------------------------
# What a pass has to move and compute

def work(case):
    op, e = case["op"], 4 if case.get("dtype") == "f32" else 2
    if op == "extend":
        new = _new_lengths(case)
        lens, bs = _lengths(case), case["bs"]
        T = sum(max(0, n) for n in new) + case["pad"]
        taken = sum((c + max(0, n) + bs - 1) // bs - (c + bs - 1) // bs for c, n in zip(lens, new))
        back = sum((c + bs - 1) // bs for c, n in zip(lens, new) if n < 0)
        # positions and slots written; the tail blocks read; lengths in and out; queue entries moved
        return {"bytes": T * 12 + case["B"] * (4 + 4 + 4 + 4 + 4) + (taken + back) * 8, "flops": T * 4}
    if op == "rope":
        T, D = case["T"], case["D"]
        n = T * (case["Hq"] + 2 * case["Hkv"]) * D
        return {"bytes": 2 * n * e + T * 12 + case["rd"] * 2,
                "flops": 3 * T * (case["Hq"] + case["Hkv"]) * case["rd"]}
    if op == "append4":
        n = 2 * case["T"] * case["Hkv"] * case["D"]
        # the 16-bit rows in, the 4-bit ones out; and back
        return {"bytes": 2 * (n * 2 + n * 9 / 16) + 16 * case["T"], "flops": 6 * n}
    seen = sum(_visible(case))
    per = case["D"] * 9 / 16 if op == "decode4" else case["D"] * e
    return {"bytes": seen * case["Hkv"] * per * 2 + 2 * case["B"] * case["Hq"] * case["D"] * e +
            seen / case["bs"] * 4 + case["B"] * 4,
            "flops": 4 * seen * case["Hq"] * case["D"]}


# ---------------------------------------------------------------------------
# The definitions in 64 bits

def exact(case, seed):
    op = case["op"]
    if op == "extend":
        return None
    st = prepare(case, seed)
    if op == "rope":
        ang = np.outer(st["positions"].cpu().numpy().astype(np.float64),
                       st["inv_freq"].cpu().numpy().astype(np.float64))
        c, s = np.cos(ang) * st["mscale"], np.sin(ang) * st["mscale"]
        half, rd = case["rd"] // 2, case["rd"]

        def turned(x):
            x = x.double().cpu().numpy().copy()
            for i in range(half):
                a, b = (i, i + half) if case["layout"] == "half" else (2 * i, 2 * i + 1)
                xa, xb = x[:, :, a].copy(), x[:, :, b].copy()
                x[:, :, a] = xa * c[:, None, i] - xb * s[:, None, i]
                x[:, :, b] = xb * c[:, None, i] + xa * s[:, None, i]
            return torch.from_numpy(x)

        pools = []
        where = st["slots"].cpu()
        for pool, x in ((st["k_pool"], turned(st["k"])), (st["v_pool"], st["v"].double().cpu())):
            flat = pool.double().cpu().transpose(1, 2).reshape(-1, case["Hkv"], case["D"])
            flat[where] = x
            pools.append(flat.view(-1, case["bs"], case["Hkv"], case["D"]).transpose(1, 2).contiguous())
        assert rd <= case["D"]
        return [turned(st["q"]), pools[0], pools[1]]
    if op == "append4":
        out = []
        for x in (st["k"], st["v"]):
            g = x.double().reshape(x.shape[0], case["Hkv"], case["D"] // 64, 64)
            lo, hi = g.min(-1, keepdim=True).values, g.max(-1, keepdim=True).values
            step = ((hi - lo) / 15).to(torch.bfloat16).double()
            n = torch.clamp(torch.round(torch.where(step > 0, (g - lo) / step, 0.0)), 0, 15)
            out.append((lo + step * n).reshape(x.shape))
        return out
    B, Hq, Hkv, D, bs, W, S = (case[x] for x in ("B", "Hq", "Hkv", "D", "bs", "window", "sinks"))
    G = Hq // Hkv
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device=DEV)
    for s, n in enumerate(_lengths(case)):
        t = torch.arange(n, device=DEV)
        if W:
            t = t[(t >= n - W) | (t < S)]
        block, tok = st["tables"][s].long()[t // bs], t % bs
        rows = []
        for pool, value in ((st["k_pool"], False), (st["v_pool"], True)):
            if op == "sinks":
                rows.append(pool[block, :, tok].double())
                continue
            sub = pool.view(pool.shape[0], Hkv, bs // 16, 9 * D)[block, :, tok // 16]
            at = code_places(D, value)[tok % 16] + (tok % 16)[:, None] * D
            byte = torch.gather(sub, 2, (at // 2)[:, None].expand(-1, Hkv, -1))
            code = torch.where((at % 2)[:, None] == 1, byte // 16, byte % 16).double()
            pair = sub[:, :, 8 * D:].contiguous().view(torch.bfloat16).double().view(len(t), Hkv, 16, D // 64, 2)
            pair = pair[torch.arange(len(t), device=DEV), :, tok % 16].repeat_interleave(64, 2)
            rows.append(pair[..., 1] + pair[..., 0] * code)
        q = st["q"][s].double().view(Hkv, G, D)
        w = torch.softmax(st["scale"] * torch.einsum("hgd,thd->hgt", q, rows[0]), -1)
        out[s] = torch.einsum("hgt,thd->hgd", w, rows[1]).reshape(Hq, D)
    return out
