"""NaN and infinities among queries and keys, in every way in which the 4-bit
decode and the windowed decode with sinks cut a batch: pieces of a sequence
merged in a CTA, one warp a sequence, equal runs with the merge kernel.

By the definition, a head's output is NaN as soon as one visible logit is NaN
(whatever the others are), and every other row is what it is without the NaN,
bit for bit. The batches are sized by the device's multiprocessors so that each
way is taken: a few sequences (many pieces each), nearly a wave of warps (one
each), more sequences than a wave holds."""

import numpy as np
import pytest
import torch

from oracle import attention_definition
from paged_kv_cache_336_b200 import binding

from gpu_util import BF16_MAX_ABS, F32_MAX_ABS, to_f64

pytestmark = pytest.mark.gpu

BS, MBS, CTX = 16, 32, 177                 # 12 units, the last holds one token
BLOCKS = 12                                # of a sequence
WAYS = ["pieces", "whole", "runs"]
PARTITION = {"pieces": 512, "whole": 512, "runs": 32}  # (many small partitions ask for equal runs)


def num_seqs(way, warps, lists):
    """Sequences that the rule cuts in this way, with at most `warps` warps per
    multiprocessor at work."""
    wave = torch.cuda.get_device_properties(0).multi_processor_count * warps
    n = {"pieces": 8, "whole": max(8, wave * 3 // (4 * lists)), "runs": min(4096, 2 * wave // lists + 200)}[way]
    assert way != "runs" or n * lists > wave
    return n


def batch(num):
    """Block tables of `num` sequences of CTX tokens, the first eight with blocks of
    their own, the others sharing one set; sequence 5 is empty."""
    tables = np.full((num, MBS), -1, dtype=np.int32)
    own = np.random.default_rng(1).permutation(9 * BLOCKS).reshape(9, BLOCKS)
    for s in range(num):
        tables[s, :BLOCKS] = own[min(s, 8)]
    lens = np.full(num, CTX, dtype=np.int32)
    lens[5] = 0
    return torch.from_numpy(tables).cuda(), torch.from_numpy(lens).cuda(), own


def slots_of(own, s, tokens):
    t = np.asarray(list(tokens))
    return own[s][t // BS] * BS + t % BS


# tokens whose keys hold a NaN, by sequence; in sequence 0 a query does
BAD_KEYS = {1: [CTX - 1], 2: range(CTX), 3: [0], 6: range(5 * 16, 6 * 16), 7: [3, 90]}


def expect(got, clean, Hq, heads, bad_q):
    """Rows that must be NaN: sequence 0's head `bad_q`, and in the sequences with a
    bad key the query heads of the first KV head (`heads` of them)."""
    nan = torch.zeros(got.shape[:2], dtype=torch.bool, device="cuda")
    nan[0, bad_q] = True
    for s in BAD_KEYS:
        nan[s, :heads] = True
    assert torch.isnan(got[nan]).all(), torch.isnan(got).all(-1)[:8].int()
    assert torch.equal(got[~nan], clean[~nan])
    assert torch.all(clean[5] == 0) and torch.isfinite(clean).all()


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("D,Hq,Hkv", [(64, 4, 2), (128, 8, 1), (128, 18, 2), (256, 2, 1)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 4)])
def test_4bit_decode(D, Hq, Hkv, way, window, sinks):
    warps = 8 if D == 256 else 12
    num = num_seqs(way, warps, Hkv * (-(-(Hq // Hkv) // 8)))
    tables, lens, own = batch(num)
    g = torch.Generator(device="cuda").manual_seed(D + Hq)
    rows = [torch.randn(9 * BLOCKS * BS, Hkv, D, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2)]
    q = torch.randn(num, Hq, D, device="cuda", generator=g).to(torch.bfloat16)
    every = torch.arange(9 * BLOCKS * BS, device="cuda")

    def call(q, k):
        pools = binding.q4_pools(9 * BLOCKS, Hkv, BS, D)
        binding.kv_append_q4(k, rows[1], every, *pools)
        return binding.decode_q4(q, *pools, tables, lens, 0.1, window=window, sinks=sinks,
                                 partition_tokens=PARTITION[way])

    clean = call(q, rows[0])
    visible = [t for t in range(CTX) if not window or t >= CTX - window or t < sinks]
    for what, bad_q in ((float("nan"), Hq - 1), (float("inf"), 0)):
        q2, k2 = q.clone(), rows[0].clone()
        q2[0, bad_q, D // 2 + 1] = what
        for s, tokens in BAD_KEYS.items():
            assert set(tokens) & set(visible)
            k2[torch.from_numpy(slots_of(own, s, tokens)).cuda(), 0, D - 1] = what
        expect(call(q2, k2), clean, Hq, Hq // Hkv, bad_q)


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("dtype,D,Hq,Hkv", [(torch.float32, 64, 4, 2), (torch.float32, 128, 8, 1),
                                            (torch.bfloat16, 64, 8, 2), (torch.bfloat16, 128, 16, 1),
                                            (torch.bfloat16, 256, 2, 1)])
@pytest.mark.parametrize("window,sinks", [(100, 4), (10_000, 0)])
def test_windows_with_sinks(dtype, D, Hq, Hkv, way, window, sinks):
    # the rings leave room for 8 (head_dim 128) to 24 (64) warps a multiprocessor
    num = num_seqs(way, 24 if way == "runs" else 8, Hkv)
    tables, lens, own = batch(num)
    g = torch.Generator(device="cuda").manual_seed(D + Hq)
    k, v = (torch.randn(9 * BLOCKS, Hkv, BS, D, device="cuda", generator=g).to(dtype) for _ in range(2))
    q = torch.randn(num, Hq, D, device="cuda", generator=g).to(dtype)

    def call(q, k):
        return binding.decode_split_sinks(q, k, v, tables, lens, 0.1, window, sinks, partition_tokens=PARTITION[way])

    clean = call(q, k)
    q2, k2 = q.clone(), k.clone()
    q2[0, Hq - 1, D // 2 + 1] = float("nan")
    for s, tokens in BAD_KEYS.items():
        slot = torch.from_numpy(slots_of(own, s, tokens)).cuda()
        k2[slot // BS, 0, slot % BS, D - 1] = float("nan")
    expect(call(q2, k2), clean, Hq, Hq // Hkv, Hq - 1)


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("dtype,D,Hq,Hkv", [(torch.float32, 64, 4, 2), (torch.bfloat16, 64, 8, 2),
                                            (torch.bfloat16, 128, 16, 1)])
@pytest.mark.parametrize("window,sinks", [(100, 4), (10_000, 0)])
def test_logits_of_minus_infinity_weigh_nothing(dtype, D, Hq, Hkv, way, window, sinks):
    """Keys that make every head's logit -inf, where BAD_KEYS has them: the softmax of
    the others; nothing but such logits (sequence 2): zeros."""
    num = num_seqs(way, 24 if way == "runs" else 8, Hkv)
    tables, lens, own = batch(num)
    g = torch.Generator(device="cuda").manual_seed(D + Hq)
    k, v = (torch.randn(9 * BLOCKS, Hkv, BS, D, device="cuda", generator=g).to(dtype) for _ in range(2))
    q = torch.randn(num, Hq, D, device="cuda", generator=g).to(dtype)
    q[..., D - 1] = q[..., D - 1].abs() + 0.5
    for s, tokens in BAD_KEYS.items():
        slot = torch.from_numpy(slots_of(own, s, tokens)).cuda()
        k[slot // BS, :, slot % BS, D - 1] = -float("inf")
    got = to_f64(binding.decode_split_sinks(q, k, v, tables, lens, 0.1, window, sinks,
                                            partition_tokens=PARTITION[way])[:9])
    assert np.all(np.isfinite(got)) and np.all(got[2] == 0) and np.all(got[5] == 0)
    t = np.arange(CTX)
    for s in (0, 1, 3, 4, 6, 7):
        see = (t >= CTX - window) | (t < sinks)
        see[list(BAD_KEYS.get(s, []))] = False
        slot = slots_of(own, s, t[see])
        K, V = (to_f64(x)[slot // BS, :, slot % BS] for x in (k, v))
        for h in range(Hq):
            want = attention_definition(to_f64(q[s, h]), K[:, h // (Hq // Hkv)], V[:, h // (Hq // Hkv)], 0.1)
            limit = F32_MAX_ABS if dtype == torch.float32 else BF16_MAX_ABS
            assert np.abs(got[s, h] - want).max() <= limit, (s, h)
