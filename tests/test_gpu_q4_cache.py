"""pa_kv_append_q4 and pa_kv_gather_q4: the pools' bytes and the values read
back are compared exactly with the oracle's quantisation and layout."""

import numpy as np
import pytest
import torch

import oracle
from paged_kv_cache_336_b200 import binding

pytestmark = pytest.mark.gpu


def rows(seed, T, H, D, kind):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, H, D, device="cuda", generator=g)
    if kind == "wide":        # channels of very different sizes
        x = x * torch.exp(4 * torch.randn(H, D, device="cuda", generator=g))
    elif kind == "grid":      # whole numbers: exact ties between codes are common
        x = torch.randint(-30, 31, (T, H, D), device="cuda", generator=g).float()
    elif kind == "tiny":      # scales among the subnormal numbers
        x = x * 2.0 ** -126
    elif kind == "huge":      # max - min overflows fp32
        x = (x * 1e38).clamp(-3.3e38, 3.3e38)
    elif kind == "flat":
        x = torch.full_like(x, -1.5)
    return x.to(torch.bfloat16)


def append(k, v, slots, NB, H, bs, D, err=None):
    kp, vp = binding.q4_pools(NB, H, bs, D)
    kp.fill_(0xA5)
    vp.fill_(0x5A)
    binding.kv_append_q4(k, v, slots, kp, vp, dev_err=err)
    return kp, vp


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("bs", [16, 32])
@pytest.mark.parametrize("kind", ["normal", "wide", "grid", "tiny", "huge", "flat"])
def test_pool_bytes_and_values(D, bs, kind):
    T, H = 41, 3
    k, v = rows(1, T, H, D, kind), rows(2, T, H, D, kind)
    NB = 5
    slots = torch.randperm(NB * bs, device="cuda")[:T]
    slots[4] = -7
    kp, vp = append(k, v, slots, NB, H, bs, D)
    sl = slots.cpu().numpy()
    for pool, x, fill, value in ((kp, k, 0xA5, False), (vp, v, 0x5A, True)):
        want = np.full(tuple(pool.shape), fill, dtype=np.uint8)
        oracle.q4_write(want, x.float().cpu().numpy(), sl, bs, value)
        assert np.array_equal(pool.cpu().numpy(), want)
    keep = [t for t in range(T) if sl[t] >= 0]
    for dtype in (torch.float32, torch.bfloat16):
        out = (torch.full((T, H, D), 9.0, dtype=dtype, device="cuda"),
               torch.full((T, H, D), 9.0, dtype=dtype, device="cuda"))
        binding.kv_gather_q4(kp, vp, slots, D, out=out)
        for got, pool, value in zip(out, (kp, vp), (False, True)):
            want = oracle.q4_read(pool.cpu().numpy(), sl[keep], D, bs, value)
            # fp32: one fused multiply-add, half a step; bf16: that and half a step more
            tol = np.abs(want) * (2.0 ** -24 if dtype == torch.float32 else 2.0 ** -8 + 2.0 ** -23) + 1e-45
            if kind == "tiny":
                tol = tol + (2.0 ** -149 if dtype == torch.float32 else 2.0 ** -133)
            assert np.all(np.abs(got[keep].double().cpu().numpy() - want) <= tol)
            assert torch.all(got[4] == 9.0)


def test_non_finite_groups_read_nan_and_spare_their_neighbours():
    D, bs = 128, 16
    k = rows(3, 6, 1, D, "normal")
    k[1, 0, 5] = float("nan")
    k[2, 0, 100] = float("inf")
    k[3, 0, 0] = float("-inf")
    slots = torch.arange(6, device="cuda") + 9
    kp, vp = append(k, k, slots, 2, 1, bs, D)
    a, b = binding.kv_gather_q4(kp, vp, slots, D)
    for x in (a, b):
        nan = torch.isnan(x[:, 0]).view(6, 2, 64)
        want = torch.zeros(6, 2, dtype=torch.bool, device="cuda")
        want[1, 0] = want[2, 1] = want[3, 0] = True
        assert torch.equal(nan.all(-1), want) and torch.equal(nan.any(-1), want)


def test_views_of_a_fused_product():
    T, H, D, bs = 33, 2, 128, 16
    x = rows(4, T, 6 * H, D, "wide").view(T, -1)
    k, v = (x[:, i * H * D:(i + 1) * H * D].unflatten(1, (H, D)) for i in (2, 4))
    slots = torch.randperm(64, device="cuda")[:T]
    a = append(k, v, slots, 4, H, bs, D)
    b = append(k.contiguous(), v.contiguous(), slots, 4, H, bs, D)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_bad_slots_and_repeated_reads():
    T, H, D, bs, NB = 10, 2, 64, 32, 3
    k = rows(5, T, H, D, "normal")
    slots = torch.arange(T, device="cuda")
    slots[2] = NB * bs
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kp, vp = append(k, k, slots, NB, H, bs, D, err)
    assert int(err.item()) == binding.DEVERR_SLOT
    assert torch.all(kp[1:] == 0xA5)
    err.zero_()
    again = torch.tensor([0, 0, 1, 1 << 50, 0, -1], device="cuda")
    out = torch.zeros(2, 6, H, D, dtype=torch.bfloat16, device="cuda")
    a, _ = binding.kv_gather_q4(kp, vp, again, D, out=(out[0], out[1]), dev_err=err)
    assert int(err.item()) == binding.DEVERR_SLOT
    assert torch.equal(a[0], a[1]) and torch.equal(a[0], a[4]) and torch.all(a[3] == 0) and torch.all(a[5] == 0)


def test_blocks_copy_and_swap_as_they_are():
    """The 4-bit pools go through copy_blocks and the swaps like any other."""
    T, H, D, bs, NB = 48, 2, 128, 16, 6
    k, v = rows(6, T, H, D, "normal"), rows(7, T, H, D, "normal")
    kp, vp = append(k, v, torch.arange(T, device="cuda"), NB, H, bs, D)
    binding.copy_blocks(kp, vp, torch.tensor([[0, 4], [2, 5]], device="cuda"))
    assert torch.equal(kp[4], kp[0]) and torch.equal(vp[5], vp[2])
    hk, hv = (torch.zeros(2, *kp.shape[1:], dtype=torch.uint8).pin_memory() for _ in range(2))
    binding.swap_out(kp, vp, hk, hv, torch.tensor([[1, 1]], device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(hk[1], kp[1].cpu()) and torch.equal(hv[1], vp[1].cpu())
    binding.swap_in(hk, hv, kp, vp, torch.tensor([[1, 3]], device="cuda"))
    assert torch.equal(kp[3], kp[1]) and torch.equal(vp[3], vp[1])


def test_zero_tokens():
    kp, vp = binding.q4_pools(2, 1, 16, 64)
    e = torch.empty(0, 1, 64, dtype=torch.bfloat16, device="cuda")
    s = torch.empty(0, dtype=torch.int64, device="cuda")
    binding.kv_append_q4(e, e, s, kp, vp)
    a, b = binding.kv_gather_q4(kp, vp, s, 64)
    assert a.shape == (0, 1, 64) and int(kp.sum()) == 0
