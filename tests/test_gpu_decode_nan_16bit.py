"""NaN among queries and keys in pa_decode, pa_decode_split and the windowed
split decode: a head's output is NaN as soon as one visible logit is NaN (whole
partitions of NaN logits, all of a CTA's warps), and every other row is what it
is without it, bit for bit."""

import os

import pytest
import torch

from paged_kv_cache_336_b200 import binding

pytestmark = pytest.mark.gpu

BS, CTX, MBS = 16, 300, 19
CALLS = {
    "decode": lambda *a: binding.decode(*a),
    "split": lambda *a: binding.decode_split(*a, partition_tokens=64),
    "window": lambda *a: binding.decode_split_window(*a, window=200, partition_tokens=64),
}


@pytest.mark.parametrize("split_kernel", ["ticket", "stream"])
@pytest.mark.parametrize("call", list(CALLS))
@pytest.mark.parametrize("dtype,D,Hq,Hkv", [(torch.float32, 64, 4, 2), (torch.float32, 128, 2, 2),
                                            (torch.bfloat16, 128, 8, 1), (torch.bfloat16, 64, 4, 4)])
def test_a_nan_reaches_its_head(dtype, D, Hq, Hkv, call, split_kernel):
    g = torch.Generator(device="cuda").manual_seed(D + Hq)
    B = 5
    k, v = (torch.randn(B * MBS, Hkv, BS, D, device="cuda", generator=g).to(dtype) for _ in range(2))
    q = torch.randn(B, Hq, D, device="cuda", generator=g).to(dtype)
    tables = torch.randperm(B * MBS, device="cuda", generator=g).to(torch.int32).view(B, MBS)
    lens = torch.full((B,), CTX, dtype=torch.int32, device="cuda")
    os.environ["PAGEDKV_SPLIT_KERNEL"] = split_kernel
    try:
        clean = CALLS[call](q, k, v, tables, lens, 0.1)
        q2, k2 = q.clone(), k.clone()
        q2[0, Hq - 1, 3] = float("nan")
        # sequence 1: a partition of 64 tokens; 2: everything; 3: the newest token
        for s, tokens in ((1, range(128, 192)), (2, range(CTX)), (3, [CTX - 1])):
            t = torch.tensor(list(tokens), device="cuda")
            k2[tables[s].long()[t // BS], 0, t % BS, D - 1] = float("nan")
        got = CALLS[call](q2, k2, v, tables, lens, 0.1)
    finally:
        os.environ.pop("PAGEDKV_SPLIT_KERNEL", None)
    nan = torch.zeros(B, Hq, dtype=torch.bool, device="cuda")
    nan[0, Hq - 1] = True
    nan[1:4, :Hq // Hkv] = True
    assert torch.isfinite(clean).all()
    assert torch.isnan(got[nan]).all()
    assert torch.equal(got[~nan], clean[~nan])
