"""Plain statements of the operators around a decode step: attention over the
visible tokens of a window with sinks, the 4-bit cache's quantisation and byte
layout, rotary positions, and a step's block-table bookkeeping. Written as
their definitions, one element or one token at a time where that is clearest.

The 4-bit layout is stated here from include/pagedkv.h's text (word offsets per
8 dims), independently of the kernels' index arithmetic.
"""

from __future__ import annotations

import numpy as np

from .paged_attention import attention_definition, gather_sequence


def paged_decode_sinks(q, k_pool, v_pool, block_tables, context_lens, scale: float, window: int,
                       sinks: int) -> np.ndarray:
    """Decode attention over tokens t < ctx with t >= ctx - window or t < sinks,
    float64 [num_seqs, num_q_heads, head_dim]. window 0: the whole context."""
    q = np.asarray(q)
    B, Hq, D = q.shape
    group = Hq // np.asarray(k_pool).shape[1]
    out = np.zeros((B, Hq, D), dtype=np.float64)
    for s in range(B):
        ctx = int(context_lens[s])
        t = np.arange(ctx)
        see = np.ones(ctx, dtype=bool) if window == 0 else (t >= ctx - window) | (t < sinks)
        # blocks without a visible token may be released (-1): read block 0 in their place
        row = np.maximum(np.asarray(block_tables[s]), 0)
        for h in range(Hq):
            K = gather_sequence(k_pool, row, ctx, h // group)[see]
            V = gather_sequence(v_pool, row, ctx, h // group)[see]
            out[s, h] = attention_definition(q[s, h], K, V, scale)
    return out


# ---------------------------------------------------------------------------
# 4-bit cache

def bf16_bits(x) -> np.ndarray:
    """fp32 -> bf16 bit patterns (uint16), round to nearest even; NaN -> 0x7fff."""
    u = np.asarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7fff + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(np.asarray(x, dtype=np.float32)), np.uint16(0x7fff), r)


def bf16_value(bits) -> np.ndarray:
    """bf16 bit patterns -> fp32 values."""
    return (np.asarray(bits).astype(np.uint32) << 16).view(np.float32)


def q4_quantize(x):
    """x [..., D] (bf16 values as fp32): codes uint8 [..., D], scales and minima
    as bf16 bits [..., D / 64]. mn = min, s = bf16((max - mn) / 15), code =
    rint((x - mn) / s) clamped to 0..15 in fp32; 0 where s = 0. A group with a
    NaN or an infinity: s = mn = NaN, codes 0."""
    x = np.asarray(x, dtype=np.float32)
    g = x.reshape(*x.shape[:-1], -1, 64)
    with np.errstate(all="ignore"):
        mn, mx = g.min(-1), g.max(-1)
        s_bits = bf16_bits((mx / np.float32(2) - mn / np.float32(2)) / np.float32(7.5))
        s = bf16_value(s_bits)
        # halves on both sides: the same quotient, and no overflow of the difference
        half = (g / np.float32(2) - mn[..., None] / np.float32(2)) / (s[..., None] / np.float32(2))
        code = np.rint(np.minimum(half, np.float32(15)))
    finite = np.isfinite(g).all(-1)
    code = np.where((s[..., None] > 0) & finite[..., None], code, 0).astype(np.uint8)
    nan = np.uint16(0x7fff)
    return (code.reshape(x.shape), np.where(finite, s_bits, nan),
            np.where(finite, bf16_bits(mn), nan))


def q4_word_offset(row: int, c: int, head_dim: int, value: bool) -> int:
    """Byte offset in a code row of the 32-bit word of dims 8 c .. 8 c + 7."""
    i, t, w = c // 8, (c // 2) % 4, 2 * (c // 8) + c % 2
    if not value:
        return {64: 8 * t + 4 * w, 128: 16 * t + 4 * w,
                256: 64 * ((w // 4) ^ (row % 2)) + 16 * t + 4 * (w % 4)}[head_dim]
    g = c % 8
    return {64: 4 * g, 128: 8 * (g ^ (4 * ((row // 2) % 2))) + 4 * i,
            256: 16 * (g ^ (2 * (row % 4))) + 4 * i}[head_dim]


def _q4_places(slot: int, head: int, num_kv_heads: int, block_size: int, head_dim: int):
    """(byte of the slot's code row, byte of its params, row of the sub-tile)."""
    tile = block_size // 16 * 9 * head_dim
    tok = slot % block_size
    sub = ((slot // block_size) * num_kv_heads + head) * tile + tok // 16 * 9 * head_dim
    r = tok % 16
    return sub + r * head_dim // 2, sub + 8 * head_dim + r * head_dim // 16, r


def q4_write(pool, x, slots, block_size: int, value: bool) -> None:
    """Quantises rows x [T, Hkv, D] into a pool uint8 [NB, Hkv, tile], in place;
    negative slots and slots past the pool write nothing."""
    T, H, D = x.shape
    code, s, mn = q4_quantize(x)
    flat = pool.reshape(-1)
    for t in range(T):
        slot = int(slots[t])
        if slot < 0 or slot >= pool.shape[0] * block_size:
            continue
        for h in range(H):
            row, par, r = _q4_places(slot, h, H, block_size, D)
            for c in range(D // 8):
                w = 0
                for j in range(8):
                    w |= int(code[t, h, 8 * c + j]) << (4 * j)
                at = row + q4_word_offset(r, c, D, value)
                flat[at:at + 4] = np.frombuffer(np.uint32(w).tobytes(), dtype=np.uint8)
            pairs = np.stack([s[t, h], mn[t, h]], -1).astype(np.uint16)
            flat[par:par + D // 16] = pairs.reshape(-1).view(np.uint8)


def q4_read(pool, slots, head_dim: int, block_size: int, value: bool) -> np.ndarray:
    """Values mn + s * code of the slots' rows, float64 [T, Hkv, D]."""
    D, H = head_dim, pool.shape[1]
    flat = pool.reshape(-1)
    out = np.zeros((len(slots), H, D), dtype=np.float64)
    for t, slot in enumerate(slots):
        for h in range(H):
            row, par, r = _q4_places(int(slot), h, H, block_size, D)
            pair = bf16_value(flat[par:par + D // 16].copy().view(np.uint16)).astype(np.float64)
            for c in range(D // 8):
                at = row + q4_word_offset(r, c, D, value)
                w = int(flat[at:at + 4].copy().view(np.uint32)[0])
                for j in range(8):
                    out[t, h, 8 * c + j] = pair[2 * (c // 8) + 1] + pair[2 * (c // 8)] * ((w >> (4 * j)) & 15)
    return out


def q4_dense(pool, head_dim: int, block_size: int, value: bool) -> np.ndarray:
    """A whole pool as [NB, Hkv, block_size, D] values (for the paged oracles)."""
    NB, H = pool.shape[:2]
    v = q4_read(pool, np.arange(NB * block_size), head_dim, block_size, value)
    return v.reshape(NB, block_size, H, head_dim).transpose(0, 2, 1, 3)


# ---------------------------------------------------------------------------
# Rotary positions

def rope(x, positions, inv_freq, interleaved: bool, mscale: float) -> np.ndarray:
    """x [T, H, D] with its first 2 len(inv_freq) dims rotated, float64."""
    y = np.asarray(x, dtype=np.float64).copy()
    half = len(inv_freq)
    for t in range(y.shape[0]):
        for i in range(half):
            f = float(positions[t]) * float(inv_freq[i])
            c, s = mscale * np.cos(f), mscale * np.sin(f)
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            xa, xb = y[t, :, a].copy(), y[t, :, b].copy()
            y[t, :, a] = c * xa - s * xb
            y[t, :, b] = c * xb + s * xa
    return y


# ---------------------------------------------------------------------------
# A step's bookkeeping

def extend_tables(block_tables, context_lens, new_lens, free_list, block_size: int):
    """One step, one sequence after the other. free_list: the free blocks in
    queue order (a list). Returns (tables, lengths, query_start, positions,
    slots, free list after), or None when the blocks do not suffice. Blocks of
    leaving sequences join the queue's end after every sequence has taken its
    own; entries of -1 are passed over."""
    tables = np.array(block_tables, dtype=np.int64)
    free, back = list(free_list), []
    lens, start, pos, slots = [], [0], [], []
    for s in range(len(context_lens)):
        ctx, new = int(context_lens[s]), int(new_lens[s])
        if new < 0:
            have = -(-ctx // block_size)
            back += [int(b) for b in tables[s, :have] if b != -1]
            lens.append(0)
            start.append(start[-1])
            continue
        for p in range(ctx, ctx + new):
            b = p // block_size
            if p % block_size == 0:
                if not free:
                    return None
                tables[s, b] = free.pop(0)
            pos.append(p)
            slots.append(int(tables[s, b]) * block_size + p % block_size)
        lens.append(ctx + new)
        start.append(start[-1] + new)
    return tables, lens, start, pos, slots, free + back
