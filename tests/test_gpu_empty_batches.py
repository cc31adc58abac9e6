"""A serving step without sequences or tokens: every call of it returns, and
writes nothing."""

import pytest
import torch

from paged_kv_cache_336_b200 import binding

pytestmark = pytest.mark.gpu

HQ, HKV, D, BS, NB = 4, 2, 64, 16, 8


def test_a_step_of_nothing():
    i32 = dict(dtype=torch.int32, device="cuda")
    bf = dict(dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, **i32)
    queue = torch.arange(NB, **i32)
    tables = torch.empty(0, 3, **i32)
    step = binding.extend_tables(tables, torch.empty(0, **i32), torch.empty(0, **i32), queue,
                                 torch.tensor([2, 5], **i32), BS, 0, dev_err=err)
    assert step.query_start.tolist() == [0] and step.queue_state.tolist() == [2, 5]
    inv, m = binding.rope_frequencies(D)
    k16, v16 = (torch.ones(NB, HKV, BS, D, **bf) for _ in range(2))
    k4, v4 = binding.q4_pools(NB, HKV, BS, D)
    new = torch.empty(0, HKV, D, **bf)
    for pools in ((k16, v16), (k4, v4)):
        q = binding.rope_append(torch.empty(0, HQ, D, **bf), new, new, step.positions, inv, step.slot_mapping, *pools,
                                mscale=m, dev_err=err)
        assert q.shape == (0, HQ, D)
    binding.kv_append_q4(new, new, step.slot_mapping, k4, v4, dev_err=err)
    assert binding.kv_gather_q4(k4, v4, step.slot_mapping, D, dev_err=err)[0].shape == (0, HKV, D)
    assert binding.decode_q4(q, k4, v4, tables, step.context_lens, 0.1, dev_err=err).shape == (0, HQ, D)
    assert binding.decode_split_sinks(q, k16, v16, tables, step.context_lens, 0.1, 32, 4,
                                      dev_err=err).shape == (0, HQ, D)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and torch.all(k16 == 1) and torch.all(k4 == 0)
