"""Pins of oracle/serving_ops.py against something other than itself (CPU):
library routines, closed forms, other oracle functions, hand-worked cases."""

import numpy as np
import pytest
import torch

import oracle
from oracle import serving_ops as so


def _batch(rng, B, Hq, Hkv, D, bs, lens):
    mbs = max(1, max(-(-n // bs) for n in lens))
    tables = np.full((B, mbs), -1, dtype=np.int32)
    ids = rng.permutation(B * mbs + 2)
    k = 0
    for s, n in enumerate(lens):
        for i in range(-(-n // bs)):
            tables[s, i] = ids[k]
            k += 1
    pool = (B * mbs + 2, Hkv, bs, D)
    return tables, rng.standard_normal(pool), rng.standard_normal(pool), rng.standard_normal((B, Hq, D))


@pytest.mark.parametrize("window,sinks", [(0, 0), (3, 0), (3, 2), (5, 4), (3, 40), (100, 1), (1, 1)])
def test_sinks_against_a_masked_library_softmax(window, sinks):
    rng = np.random.default_rng(window * 50 + sinks)
    lens = [0, 1, 7, 16, 33]
    tables, k, v, q = _batch(rng, 5, 4, 2, 8, 16, lens)
    got = oracle.paged_decode_sinks(q, k, v, tables, lens, 0.3, window, sinks)
    for s, n in enumerate(lens):
        for h in range(4):
            if n == 0:
                assert np.all(got[s, h] == 0)
                continue
            K = oracle.paged_attention.gather_sequence(k, tables[s], n, h // 2)
            V = oracle.paged_attention.gather_sequence(v, tables[s], n, h // 2)
            x = torch.from_numpy(0.3 * (K @ q[s, h]))
            for t in range(n):
                if window and t < n - window and t >= sinks:
                    x[t] = -torch.inf
            want = torch.softmax(x, 0).numpy() @ V
            np.testing.assert_allclose(got[s, h], want, atol=1e-12)
    if sinks == 0 and window:
        np.testing.assert_allclose(got, oracle.paged_decode_window(q, k, v, tables, lens, 0.3, window),
                                   atol=1e-12)


def test_bf16_rounding_against_torch():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal(4000) * np.exp(10 * rng.standard_normal(4000))).astype(np.float32)
    want = torch.from_numpy(x).to(torch.bfloat16).float().numpy()
    assert np.array_equal(so.bf16_value(so.bf16_bits(x)), want)


@pytest.mark.parametrize("scale", [1e-30, 1.0, 1e30])
def test_quantisation_error_is_at_most_half_a_step(scale):
    rng = np.random.default_rng(3)
    x = torch.from_numpy(rng.standard_normal((50, 128)) * scale).to(torch.bfloat16).float().numpy()
    code, s_bits, mn_bits = oracle.q4_quantize(x)
    s = so.bf16_value(s_bits).astype(np.float64).repeat(64, -1)
    mn = so.bf16_value(mn_bits).astype(np.float64).repeat(64, -1)
    assert code.min() == 0 and code.max() == 15
    # half a step (the rounded step ends at most 15 * 2^-8 of a step short of the
    # maximum, which is less), and the quotient's rounding to 32 bits
    err = np.abs(mn + s * code - x)
    assert np.all(err <= s * 0.5 * (1 + 2.0 ** -18))
    # the formula in torch's 32-bit arithmetic
    g = torch.from_numpy(x).view(50, 2, 64)
    lo, hi = g.amin(-1), g.amax(-1)
    if scale < 1e30:
        st = ((hi - lo) / 15).to(torch.bfloat16).float()
        assert np.array_equal(so.bf16_value(s_bits), st.numpy())
        c = torch.round((g - lo[..., None]) / st[..., None]).clamp(0, 15).view(50, 128)
        assert np.array_equal(code, c.numpy().astype(np.uint8))


def test_quantisation_special_groups():
    x = np.zeros((3, 128), dtype=np.float32)
    x[0, :64] = 2.5                       # all equal: scale 0, codes 0, value 2.5
    x[1, 3] = np.nan
    x[2, 70] = -np.inf
    code, s, mn = oracle.q4_quantize(x)
    assert np.all(code == 0)
    assert s[0, 0] == 0 and so.bf16_value(mn)[0, 0] == 2.5
    assert np.isnan(so.bf16_value(s)[1, 0]) and np.isnan(so.bf16_value(mn)[1, 0])
    assert np.isnan(so.bf16_value(s)[2, 1]) and not np.isnan(so.bf16_value(s)[2, 0])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("value", [False, True])
def test_layout_places_every_word_once_and_reads_back(D, value):
    for r in range(16):
        offs = sorted(so.q4_word_offset(r, c, D, value) for c in range(D // 8))
        assert offs == list(range(0, D // 2, 4))
    rng = np.random.default_rng(D)
    for bs in (16, 32):
        pool = rng.integers(0, 256, (3, 2, bs // 16 * 9 * D), dtype=np.uint8)
        x = torch.from_numpy(rng.standard_normal((5, 2, D))).to(torch.bfloat16).float().numpy()
        slots = np.array([0, -1, 3 * bs, bs + 15, 2 * bs + bs - 1])  # one padding, one past the pool
        before = pool.copy()
        oracle.q4_write(pool, x, slots, bs, value)
        keep = [0, 3, 4]
        code, s, mn = oracle.q4_quantize(x)
        want = so.bf16_value(mn).astype(float).repeat(64, -1) + \
            so.bf16_value(s).astype(float).repeat(64, -1) * code
        got = oracle.q4_read(pool, slots[keep], D, bs, value)
        assert np.array_equal(got, want[keep])
        # three rows of codes and parameters in two heads changed, at most
        assert (pool != before).sum() <= 3 * 2 * (D // 2 + D // 16)
        dense = oracle.q4_dense(pool, D, bs, value)
        assert np.array_equal(dense[1, :, 15], got[1])


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_is_a_complex_product(interleaved):
    rng = np.random.default_rng(5)
    x = rng.standard_normal((4, 3, 64))
    inv = 10000.0 ** (-np.arange(16) / 16)
    pos = [0, 1, 77, 100000]
    got = oracle.rope(x, pos, inv, interleaved, 1.25)
    a, b = (x[..., 0:32:2], x[..., 1:32:2]) if interleaved else (x[..., :16], x[..., 16:32])
    z = (a + 1j * b) * 1.25 * np.exp(1j * np.outer(pos, inv))[:, None]
    ga, gb = (got[..., 0:32:2], got[..., 1:32:2]) if interleaved else (got[..., :16], got[..., 16:32])
    np.testing.assert_allclose(ga + 1j * gb, z, atol=1e-10)
    assert np.array_equal(got[..., 32:], x[..., 32:])


def test_extend_tables_against_the_block_manager():
    """The same blocks, slots and queue as the reference manager's FIFO policy."""
    rng = np.random.default_rng(9)
    bs, nb, mbs = 4, 40, 12
    bm = oracle.BlockManager(nb, bs, mbs, rng.permutation(nb).tolist())
    lens = [0, 1, 4, 5, 9]
    for s, n in enumerate(lens):
        bm.allocate(s, n)
    tables = np.full((5, mbs), -1)
    for s in range(5):
        t = bm.block_table(s)
        tables[s, :len(t)] = t
    new = [3, 1, 1, -1, 8]
    got = oracle.extend_tables(tables, lens, new, list(bm.free_queue), bs)
    slots = []
    for s, n in enumerate(new):
        for _ in range(max(0, n)):
            slots.append(bm.append_slot(s).slot)
    bm.free(3)
    t, after, start, pos, sl, free = got
    # (the manager returns a sequence's blocks by id, the operator in table order)
    n = len(free) - 2
    assert sl == slots and free[:n] == list(bm.free_queue)[:n]
    assert free[n:] == tables[3, :2].tolist() and sorted(free[n:]) == list(bm.free_queue)[n:]
    assert after == [3, 2, 5, 0, 17] and start == [0, 3, 4, 5, 5, 13]
    assert pos == [0, 1, 2, 1, 4] + list(range(9, 17))
    for s in (0, 1, 2, 4):
        want = bm.block_table(s)
        assert t[s, :len(want)].tolist() == want
    assert oracle.extend_tables(tables, lens, [40, 1, 1, 1, 1], [1, 2], bs) is None
