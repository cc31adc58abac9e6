"""pa_extend_tables against the sequential statement: whole numbers, so every
output is compared exactly. Ragged batches, empty ones, padding, leaving
sequences with released blocks, rings that wrap, refusals found on the device,
graph replays."""

import random

import numpy as np
import pytest
import torch

import oracle
from paged_kv_cache_336_b200 import binding

pytestmark = pytest.mark.gpu


def build(seed, lens, new, bs, spare=7, released=(), slack=2):
    """(tables, queue, state, free list): shuffled blocks, the ring's head in its middle."""
    rng = random.Random(seed)
    rows = [n + max(0, k) for n, k in zip(lens, new)]
    mbs = max([1] + [-(-r // bs) for r in rows]) + slack
    held = sum(-(-n // bs) for n in lens)
    need = sum(-(-r // bs) for r in rows) - held
    nb = held + need + spare + 1
    ids = rng.sample(range(nb), nb)
    tables = np.full((len(lens), mbs), -1, dtype=np.int32)
    for s, n in enumerate(lens):
        for i in range(-(-n // bs)):
            tables[s, i] = ids.pop()
    free = ids
    for s, i in released:  # blocks released before a window: back in the queue already
        if tables[s, i] >= 0:
            free.append(int(tables[s, i]))
            tables[s, i] = -1
    head = (2 * nb) // 3
    queue = np.full(nb, -1, dtype=np.int32)
    for i, b in enumerate(free):
        queue[(head + i) % nb] = b
    return tables, queue, [head, len(free)], free


def cuda(x, dtype=torch.int32):
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


def call(tables, lens, new, queue, state, bs, max_tokens, err=None):
    t, q = cuda(tables), cuda(queue)
    out = binding.extend_tables(t, cuda(lens), cuda(new), q, cuda(state), bs, max_tokens, dev_err=err)
    torch.cuda.synchronize()
    return t, q, out


CASES = [
    ([5], [1], 16, 1), ([16], [1], 16, 4), ([0], [0], 16, 0), ([0, 0], [40, 33], 16, 80),
    ([15, 16, 17, 0, 31], [1, 1, 1, 1, 1], 16, 9), ([3, 40, 7], [-1, 5, -1], 16, 5),
    ([64, 64], [-1, -1], 32, 3), ([], [], 16, 0), ([], [], 16, 6), ([7], [0], 16, 3), ([1] * 300, [1] * 300, 16, 301),
]


@pytest.mark.parametrize("lens,new,bs,max_tokens", CASES)
def test_small_batches(lens, new, bs, max_tokens):
    check(1, lens, new, bs, max_tokens)


@pytest.mark.parametrize("seed,B,hi,new_hi,bs", [(0, 700, 2000, 1, 16), (1, 257, 900, 3000, 16),
                                                 (2, 4096, 64, 9, 32), (3, 33, 8192, 500, 32)])
def test_ragged_batches(seed, B, hi, new_hi, bs):
    rng = random.Random(seed)
    lens = [rng.randrange(hi) for _ in range(B)]
    new = [rng.choice([-1, 0, 1, rng.randrange(new_hi + 1)]) for _ in range(B)]
    released = [(s, i) for s in range(0, B, 3) for i in range(lens[s] // bs // 2)]
    check(seed, lens, new, bs, sum(max(0, n) for n in new) + seed * 333, released)


def check(seed, lens, new, bs, max_tokens, released=()):
    tables, queue, state, free = build(seed, lens, new, bs, released=released)
    nb = len(queue)
    want = oracle.extend_tables(tables, lens, new, free, bs)
    wt, wl, ws, wp, wsl, wfree = want
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    t, q, out = call(tables, lens, new, queue, state, bs, max_tokens, err)
    bits = int(err.item())
    # a token whose own block was released has no slot
    wsl = [x if x >= 0 else -1 for x in wsl]
    lost = any(n > 0 and lens[s] % bs and tables[s, lens[s] // bs] < 0 for s, n in enumerate(new))
    assert bits == (binding.DEVERR_BLOCK_ID if lost else 0)
    assert t.cpu().numpy().tolist() == wt.tolist()
    assert out.context_lens.tolist() == wl and out.query_start.tolist() == ws
    pad = max_tokens - len(wp)
    assert out.positions.tolist() == wp + [0] * pad
    assert out.slot_mapping.tolist() == wsl + [-1] * pad
    head, count = out.queue_state.tolist()
    assert count == len(wfree) and 0 <= head < nb
    ring = q.cpu().tolist()
    assert [ring[(head + i) % nb] for i in range(count)] == wfree


@pytest.mark.parametrize("what,bit", [
    ("blocks", binding.DEVERR_NO_FREE_BLOCKS), ("tokens", binding.DEVERR_NUM_TOKENS),
    ("head", binding.DEVERR_FREE_QUEUE), ("count", binding.DEVERR_FREE_QUEUE),
    ("room", binding.DEVERR_FREE_QUEUE), ("length", binding.DEVERR_CONTEXT_LEN),
    ("past", binding.DEVERR_CONTEXT_LEN), ("new", binding.DEVERR_CONTEXT_LEN)])
def test_nothing_changes_when_the_call_cannot_be_met(what, bit):
    lens, new, bs = [20, 33, 5], [30, 1, -1], 16
    tables, queue, state, _ = build(4, lens, new, bs)
    max_tokens = 31
    if what == "blocks":
        state[1] = 1
    elif what == "tokens":
        max_tokens = 30
    elif what == "head":
        state[0] = len(queue)
    elif what == "count":
        state[1] = -1
    elif what == "room":
        state[1] = len(queue)
    elif what == "length":
        lens[1] = -3
    elif what == "past":
        new[0] = 1000
    else:
        new[2] = -2
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    t, q, out = call(tables, lens, new, queue, state, bs, max_tokens, err)
    assert int(err.item()) == bit
    assert t.tolist() == tables.tolist() and q.tolist() == queue.tolist()
    assert out.context_lens.tolist() == lens and out.queue_state.tolist() == state
    assert out.query_start.tolist() == [0] * 4
    assert out.positions.tolist() == [0] * max_tokens and out.slot_mapping.tolist() == [-1] * max_tokens


def test_bad_queue_entries_are_reported_and_give_no_slot():
    lens, new, bs = [16, 3], [2, 1], 16
    tables, queue, state, _ = build(5, lens, new, bs)
    queue[state[0]] = 10 ** 6
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    _, _, out = call(tables, lens, new, queue, state, bs, 3, err)
    assert int(err.item()) == binding.DEVERR_BLOCK_ID
    assert out.slot_mapping.tolist() == [-1, -1, int(tables[1, 0]) * bs + 3]


def test_steps_in_a_captured_graph_follow_one_another():
    """Two calls in one graph, each reading what the other wrote: every replay
    is two decode steps; compared with the sequential statement."""
    bs, B, mbs = 16, 9, 30
    lens = [0, 5, 15, 16, 17, 31, 32, 100, 1]
    tables = np.full((B, mbs), -1, dtype=np.int32)
    ids = list(range(299, -1, -1))
    for s, n in enumerate(lens):
        for i in range(-(-n // bs)):
            tables[s, i] = ids.pop()
    t, q = cuda(tables), cuda(ids)
    a, b = binding.StepTables.empty(B, B), binding.StepTables.empty(B, B)
    a.context_lens.copy_(cuda(lens))
    a.queue_state.copy_(cuda([0, len(ids)]))
    # the ring is as long as the list of free blocks here: block ids lie beyond it
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ring = torch.full((300,), -1, dtype=torch.int32, device="cuda")
    ring[:len(ids)] = q
    one = torch.ones(B, dtype=torch.int32, device="cuda")
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=stream):
            binding.extend_tables(t, a.context_lens, one, ring, a.queue_state, bs, B, out=b, dev_err=err)
            binding.extend_tables(t, b.context_lens, one, ring, b.queue_state, bs, B, out=a, dev_err=err)
    for _ in range(20):
        g.replay()
    torch.cuda.synchronize()
    want, wl, free = tables, lens, ids
    for _ in range(40):
        want, wl, _, wp, wsl, free = oracle.extend_tables(want, wl, [1] * B, free, bs)
    assert int(err.item()) == 0
    assert a.context_lens.tolist() == wl and a.slot_mapping.tolist() == wsl and a.positions.tolist() == wp
    assert t.cpu().numpy().tolist() == want.tolist()
    assert a.queue_state.tolist()[1] == len(free)
