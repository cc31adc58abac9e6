"""The operators of a serving step run together, as a decode loop uses them:
pa_extend_tables makes blocks, positions and slots, pa_rope_append(_q4) rotates
and caches, pa_decode_split_sinks / pa_decode_q4 attends. The oracle keeps each
sequence's rotated keys and its values in plain lists and never sees a table.

Bounds. What is cached in 16 bits is the rotated key rounded once (2^-8 of it)
and the decode kernels' 2e-2 / 2e-3 of the other tests hold on top; for the
4-bit cache the oracle quantises the keys that the device cached, read back by
kv_gather_q4, so that codes cannot differ, and the same bounds hold on values of
about the same size."""

import numpy as np
import pytest
import torch

import oracle
from paged_kv_cache_336_b200 import binding

from gpu_util import BF16_MAX_ABS, BF16_MEAN_ABS, to_f64

pytestmark = pytest.mark.gpu

B, HQ, HKV, D, BS, MBS = 5, 8, 2, 128, 16, 12
NB = B * MBS + 3


class Loop:
    """Device state of a decode loop and, beside it, the oracle's."""

    def __init__(self, q4, seed):
        self.q4 = q4
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.tables = torch.full((B, MBS), -1, dtype=torch.int32, device="cuda")
        self.queue = torch.randperm(NB, device="cuda", generator=self.gen).to(torch.int32)
        self.sets = [None, None]
        self.cur = 0
        self.lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.state = torch.tensor([0, NB], dtype=torch.int32, device="cuda")
        if q4:
            self.k, self.v = binding.q4_pools(NB, HKV, BS, D)
        else:
            self.k = torch.zeros(NB, HKV, BS, D, dtype=torch.bfloat16, device="cuda")
            self.v = torch.zeros_like(self.k)
        self.inv, self.mscale = binding.rope_frequencies(64, scaling="yarn", factor=4.0)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.hist = [[] for _ in range(B)]   # slots of each sequence's tokens, in order
        self.keys = [[] for _ in range(B)]   # the oracle's rotated keys and values
        self.vals = [[] for _ in range(B)]

    def rows(self, T):
        return torch.randn(T, (HQ + 2 * HKV) * D, device="cuda", generator=self.gen).to(torch.bfloat16)

    def step(self, new, pad=0):
        """One step of `new` tokens per sequence (-1 leaves); the rotated queries
        and the step's tables."""
        T = sum(max(0, n) for n in new) + pad
        st = binding.extend_tables(self.tables, self.lens, torch.tensor(new, dtype=torch.int32, device="cuda"),
                                   self.queue, self.state, BS, T, dev_err=self.err)
        self.lens, self.state = st.context_lens, st.queue_state
        q, k, v = (x.unflatten(1, (-1, D)) for x in self.rows(T).split([HQ * D, HKV * D, HKV * D], 1))
        out = binding.rope_append(q, k, v, st.positions, self.inv, st.slot_mapping, self.k, self.v,
                                  mscale=self.mscale, dev_err=self.err)
        pos, inv = st.positions.cpu().numpy(), self.inv.cpu().numpy().astype(np.float64)
        kr = oracle.rope(to_f64(k), pos, inv, False, self.mscale)
        slots, row = st.slot_mapping.cpu().numpy(), 0
        for s, n in enumerate(new):
            if n < 0:
                self.hist[s], self.keys[s], self.vals[s] = [], [], []
            for _ in range(max(0, n)):
                assert pos[row] == len(self.keys[s])
                self.hist[s].append(int(slots[row]))
                self.keys[s].append(kr[row])
                self.vals[s].append(to_f64(v[row]))
                row += 1
        assert row == int(st.query_start[-1]) and np.all(slots[row:] == -1)
        return out, st

    def attend(self, q, window, sinks):
        scale = 1 / np.sqrt(D)
        if self.q4:
            got = binding.decode_q4(q, self.k, self.v, self.tables, self.lens, scale, window=window, sinks=sinks,
                                    partition_tokens=64, dev_err=self.err)
        else:
            got = binding.decode_split_sinks(q, self.k, self.v, self.tables, self.lens, scale, window, sinks,
                                             partition_tokens=64, dev_err=self.err)
        torch.cuda.synchronize()
        assert int(self.err.item()) == 0
        want = np.zeros((B, HQ, D))
        q64 = to_f64(q)
        for s in range(B):
            n = len(self.keys[s])
            t = np.arange(n)
            see = (t >= n - window) | (t < sinks) if window else t >= 0
            if n == 0:
                continue
            K, V = np.stack(self.keys[s]), np.stack(self.vals[s])
            if self.q4:
                kd, vd = binding.kv_gather_q4(self.k, self.v, torch.tensor(self.hist[s], device="cuda"), D,
                                              dtype=torch.float32)
                kd, vd = to_f64(kd), to_f64(vd)
                for x, y in ((kd, K), (vd, V)):  # a value is within half a step of what was cached
                    g = y.reshape(n, HKV, D // 64, 64)
                    half = (g.max(-1) - g.min(-1)) / 15 * 0.5
                    # bf16 keys (2^-8 of the largest), the step's own rounding (2^-8 over 15 steps)
                    tol = half * (1 + 2.0 ** -7) + np.abs(g).max(-1) * 2.0 ** -7
                    assert np.all(np.abs(x - y).reshape(g.shape) <= tol[..., None])
                K, V = kd, vd
            for h in range(HQ):
                want[s, h] = oracle.attention_definition(q64[s, h], K[see, h // 4], V[see, h // 4], scale)
        e = np.abs(to_f64(got) - want)
        assert e.max() <= BF16_MAX_ABS and e.mean() <= BF16_MEAN_ABS, (e.max(), e.mean())


@pytest.mark.parametrize("q4", [False, True])
def test_prefill_then_decode_then_sequences_come_and_go(q4):
    loop = Loop(q4, 1)
    loop.step([33, 1, 16, 0, 90], pad=7)              # a prefill wave with padding rows
    window, sinks = (40, 4) if not q4 else (0, 0)
    for i in range(4):
        q, _ = loop.step([1] * B)
        loop.attend(q, window, sinks)
    loop.step([-1, 0, 0, 20, 0])                      # one sequence leaves, one gets a prompt
    loop.step([50, 0, 31, 0, 0])                      # the place is taken again
    for i in range(3):
        q, _ = loop.step([1] * B)
        loop.attend(q, 24, 3)


@pytest.mark.parametrize("q4", [False, True])
def test_a_captured_step_replayed(q4):
    """extend -> rope_append -> decode in one CUDA graph of two steps: replays give
    what eager steps from the same state give, bit for bit."""
    def fresh():
        torch.manual_seed(3)
        loop = Loop(q4, 2)
        loop.step([17, 3, 40, 16, 1])
        return loop

    n_steps, scale = 12, 0.1
    rows = torch.randn(n_steps, B, (HQ + 2 * HKV) * D, device="cuda",
                       generator=torch.Generator(device="cuda").manual_seed(9)).to(torch.bfloat16)

    def one(loop, x, lens, state, out_set, attn, ws):
        st = binding.extend_tables(loop.tables, lens, torch.ones(B, dtype=torch.int32, device="cuda"), loop.queue,
                                   state, BS, B, out=out_set, dev_err=loop.err)
        q, k, v = (y.unflatten(1, (-1, D)) for y in x.split([HQ * D, HKV * D, HKV * D], 1))
        qr = binding.rope_append(q, k, v, st.positions, loop.inv, st.slot_mapping, loop.k, loop.v,
                                 mscale=loop.mscale, dev_err=loop.err)
        if q4:
            binding.decode_q4(qr, loop.k, loop.v, loop.tables, st.context_lens, scale, window=30, sinks=2,
                              workspace=ws, out=attn, dev_err=loop.err)
        else:
            binding.decode_split_sinks(qr, loop.k, loop.v, loop.tables, st.context_lens, scale, 30, 2,
                                       workspace=ws, out=attn, dev_err=loop.err)

    def run(graph):
        loop = fresh()
        ws = binding.SplitWorkspace(B, HQ, D, BS, MBS, 64)
        sets = [binding.StepTables.empty(B, B), binding.StepTables.empty(B, B)]
        sets[1].context_lens.copy_(loop.lens)
        sets[1].queue_state.copy_(loop.state)
        x = torch.empty(2, B, rows.shape[2], dtype=torch.bfloat16, device="cuda")
        attn = torch.empty(2, B, HQ, D, dtype=torch.bfloat16, device="cuda")
        outs = []

        def pair():
            for i in range(2):
                one(loop, x[i], sets[1 - i].context_lens, sets[1 - i].queue_state, sets[i], attn[i], ws)

        g = None
        if graph:
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=torch.cuda.Stream()):
                pair()
        for j in range(0, n_steps, 2):
            x.copy_(rows[j:j + 2])
            g.replay() if graph else pair()
            outs.append(attn.clone())
        torch.cuda.synchronize()
        assert int(loop.err.item()) == 0
        return torch.cat(outs), loop.tables.clone(), loop.k.clone(), sets[1].context_lens.tolist()

    a, b = run(False), run(True)
    assert a[3] == b[3] == [17 + n_steps, 3 + n_steps, 40 + n_steps, 16 + n_steps, 1 + n_steps]
    assert all(torch.equal(x, y) for x, y in zip(a[:3], b[:3]))


def test_a_4bit_sequence_laid_out_for_prefill():
    """kv_gather_q4 and kv_append bring a 4-bit sequence into 16-bit pools, over
    which pa_prefill attends a chunk of new tokens."""
    loop = Loop(True, 5)
    loop.step([60, 0, 0, 0, 0])
    slots = torch.tensor(loop.hist[0], device="cuda")
    k, v = binding.kv_gather_q4(loop.k, loop.v, slots, D)
    kp = torch.zeros(NB, HKV, BS, D, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    binding.kv_append(k, v, slots, kp, vp)
    q = torch.randn(60, HQ, D, device="cuda", generator=loop.gen).to(torch.bfloat16)
    out = binding.prefill(q, kp, vp, loop.tables[:1].contiguous(), [60], [60], 0.1, partition_tokens=64)
    want = oracle.paged_prefill(to_f64(q), to_f64(kp), to_f64(vp), loop.tables[:1].cpu().numpy(), [60], [60], 0.1)
    e = np.abs(to_f64(out) - want)
    assert e.max() <= BF16_MAX_ABS and e.mean() <= BF16_MEAN_ABS


def test_two_streams_at_once():
    """Two loops on two streams with workspaces of their own: neither disturbs the other."""
    res = []
    for both in (False, True):
        loops = [Loop(True, 11), Loop(False, 12)]
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        qs = []
        for loop in loops:
            loop.step([100, 5, 16, 31, 64])
            q, _ = loop.step([1] * B)
            qs.append(q)
        wss = [binding.SplitWorkspace(B, HQ, D, BS, MBS, 32) for _ in loops]
        torch.cuda.synchronize()
        outs = []
        for rep in range(20):
            for loop, q, ws, st in zip(loops, qs, wss, streams):
                with torch.cuda.stream(st if both else streams[0]):
                    if loop.q4:
                        outs.append(binding.decode_q4(q, loop.k, loop.v, loop.tables, loop.lens, 0.1, workspace=ws))
                    else:
                        outs.append(binding.decode_split_sinks(q, loop.k, loop.v, loop.tables, loop.lens, 0.1, 50, 4,
                                                               workspace=ws))
        torch.cuda.synchronize()
        assert all(torch.equal(o, outs[i % 2]) for i, o in enumerate(outs))
        res.append(outs[:2])
    assert all(torch.equal(x, y) for x, y in zip(*res))


def test_what_a_call_allocates_belongs_to_its_stream():
    """With `stream`, outputs and the workspace come from that stream's memory: the
    current stream's next tensors never take it while the call may still run."""
    loop = Loop(True, 13)
    q, st = loop.step([30, 5, 16, 31, 64])
    k = torch.zeros(64, HKV, D, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(64, dtype=torch.int32, device="cuda")
    slots = torch.full((64,), -1, dtype=torch.int64, device="cuda")
    pools = [torch.zeros(NB, HKV, BS, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    q1 = q[:B].contiguous()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    calls = [
        lambda: binding.SplitWorkspace(B, HQ, D, BS, MBS, 32, stream=side).buffer,
        lambda: binding.decode_q4(q1, loop.k, loop.v, loop.tables, loop.lens, 0.1, stream=side),
        lambda: binding.decode_split_sinks(q1, *pools, loop.tables, loop.lens, 0.1, 50, 4, stream=side),
        lambda: binding.kv_gather_q4(loop.k, loop.v, slots, D, stream=side)[0],
        lambda: binding.rope_append(k, k, k, pos, loop.inv, slots, *pools, stream=side),
        lambda: binding.extend_tables(loop.tables, loop.lens, zero, loop.queue, loop.state, BS, 64,
                                      stream=side).slot_mapping,
    ]
    for call in calls:
        t = call()
        at, n = t.data_ptr(), t.untyped_storage().nbytes()
        torch.cuda.synchronize()
        del t
        here = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(64)]
        assert at not in [x.data_ptr() for x in here]
        with torch.cuda.stream(side):
            there = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(64)]
        assert at in [x.data_ptr() for x in there]
