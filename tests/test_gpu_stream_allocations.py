"""Calls with a ``stream`` allocate what the caller does not give them from that
stream's memory, and a workspace's header is zeroed on the stream whose call
uses it: memory of another stream could still be in use there, or be given
away while the call runs."""

import numpy as np
import pytest
import torch

from paged_kv_cache_336_b200 import binding

pytestmark = pytest.mark.gpu

B, HQ, HKV, D, BS, MBS = 4, 8, 2, 128, 16, 8
NB = B * MBS
NO_GROUPS = (np.zeros(1, np.int32), np.zeros(0, np.int32), np.zeros(0, np.int32))


def inputs():
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(B, HQ, D, device="cuda", generator=g).to(torch.bfloat16)
    k, v = (torch.randn(NB, HKV, BS, D, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    tables = torch.arange(NB, dtype=torch.int32, device="cuda").view(B, MBS)
    lens = torch.tensor([5, 128, 77, 16], dtype=torch.int32, device="cuda")
    return q, k, v, tables, lens


CALLS = {
    "decode": lambda st, *a: binding.decode(*a, 0.1, stream=st),
    "decode_split": lambda st, *a: binding.decode_split(*a, 0.1, partition_tokens=32, stream=st),
    "decode_split_window": lambda st, *a: binding.decode_split_window(*a, 0.1, 40, partition_tokens=32, stream=st),
    "decode_shared_prefix": lambda st, *a: binding.decode_shared_prefix(*a, 0.1, NO_GROUPS, partition_tokens=32,
                                                                        stream=st),
    "prefill": lambda st, q, k, v, t, c: binding.prefill(q, k, v, t, c.tolist(), [1] * B, 0.1, stream=st),
    "prefill_workspace": lambda st, *a: binding.prefill_workspace(B, B, HQ, HKV, D, BS, MBS, 2048,
                                                                  stream=st).buffer,
    "shared_prefix_workspace": lambda st, *a: binding.shared_prefix_workspace(B, HQ, HKV, D, BS, MBS, 32,
                                                                              stream=st).buffer,
}


@pytest.mark.parametrize("name", list(CALLS))
def test_what_a_call_allocates_belongs_to_its_stream(name):
    args = inputs()
    want = CALLS[name](None, *args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    t = CALLS[name](side, *args)
    torch.cuda.synchronize()
    if not name.endswith("workspace"):
        assert torch.equal(t, want)
    at, n = t.data_ptr(), t.untyped_storage().nbytes()
    del t
    here = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(64)]
    assert at not in [x.data_ptr() for x in here]
    with torch.cuda.stream(side):
        there = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(64)]
    assert at in [x.data_ptr() for x in there]


@pytest.mark.parametrize("make", [
    lambda st: binding.Workspace(1 << 20, stream=st),
    lambda st: binding.SplitWorkspace(B, HQ, D, BS, MBS, 32, stream=st),
    lambda st: binding.prefill_workspace(B, B, HQ, HKV, D, BS, MBS, 2048, stream=st),
    lambda st: binding.shared_prefix_workspace(B, HQ, HKV, D, BS, MBS, 32, stream=st)])
def test_a_workspace_is_zeroed_on_its_stream(make):
    """The stream is still writing to the memory that the workspace will reuse."""
    side = torch.cuda.Stream()
    n = make(None).buffer.numel()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        old = torch.empty(n, dtype=torch.uint8, device="cuda")
        at = old.data_ptr()
        torch.cuda._sleep(20_000_000)  # some ten milliseconds
        old.fill_(0xff)
        del old
    ws = make(side)
    torch.cuda.synchronize()
    assert ws.buffer.data_ptr() == at
    first = ws.ptr - at
    assert torch.all(ws.buffer[first:first + 256] == 0)
