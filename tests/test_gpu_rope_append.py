"""pa_rope_append and pa_rope_append_q4 against the 64-bit definition.

Bound of the rotated values. The angle in half turns is rounded once to fp32:
at most 2^-25 of a half turn, pi 2^-25 = 9.4e-8 radians; sincospif is within 2
ulp of a value of at most 1 (2^-23), and the products with mscale round once
more (2^-24): 9.4e-8 + 1.2e-7 + 6e-8 < 2.8e-7 per unit of mscale on cos and
sin. The rotation's two products and sum round by at most 3 * 2^-24 = 1.8e-7
of |a| + |b|. Together below 5e-7 mscale (|a| + |b|); bf16 outputs add half a
step, 2^-8 of the value."""

import numpy as np
import pytest
import torch

import oracle
from oracle import serving_ops as so
from paged_kv_cache_336_b200 import binding

pytestmark = pytest.mark.gpu


def make(seed, T, Hq, Hkv, D, bs, dtype, far, fused, extra=3):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g).to(dtype)

    if fused:
        x = normal(T, (Hq + 2 * Hkv) * D)
        q, k, v = (p.unflatten(1, (-1, D)) for p in x.split([Hq * D, Hkv * D, Hkv * D], 1))
    else:
        q, k, v = normal(T, Hq, D), normal(T, Hkv, D), normal(T, Hkv, D)
    nb = -(-T // bs) + extra
    slots = torch.randperm(nb * bs, device="cuda", generator=g)[:T]
    pos = torch.randint(0, far, (T,), device="cuda", generator=g, dtype=torch.int32)
    return q, k, v, pos, slots, normal(nb, Hkv, bs, D), normal(nb, Hkv, bs, D)


def rotated_bound(x, rd, interleaved, mscale, dtype):
    """The bound above for every element of x [T, H, D] (float64 numpy)."""
    half = rd // 2
    tol = np.zeros_like(x)
    a, b = (np.arange(half) * 2, np.arange(half) * 2 + 1) if interleaved else \
        (np.arange(half), np.arange(half) + half)
    pair = np.abs(x[..., a]) + np.abs(x[..., b])
    tol[..., a] = tol[..., b] = 5e-7 * mscale * pair
    return tol


def f64(t):
    return t.double().cpu().numpy()


def check_values(got, want, tol, dtype):
    if dtype == torch.bfloat16:
        tol = tol + np.abs(want) * 2.0 ** -8 + 1e-38
    err = np.abs(f64(got) - want)
    assert np.all(err <= tol), float((err - tol).max())


SHAPES = [
    # T, Hq, Hkv, D, rotary_dim, bs
    (1, 1, 1, 64, 64, 16), (1, 32, 8, 128, 128, 16), (3, 12, 2, 64, 16, 32), (37, 4, 4, 256, 48, 16),
    (130, 8, 1, 128, 96, 32), (1201, 3, 1, 64, 32, 16), (5, 0, 2, 128, 128, 16), (9, 2, 1, 128, 0, 16),
]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("fused", [False, True])
def test_matches_definition(shape, dtype, interleaved, fused):
    T, Hq, Hkv, D, rd, bs = shape
    q, k, v, pos, slots, kp, vp = make(T + rd, T, Hq, Hkv, D, bs, dtype, 1 << 20, fused)
    inv = torch.tensor(10000.0 ** (-2.0 * np.arange(rd // 2) / max(rd, 1)), dtype=torch.float32, device="cuda")
    if T > 4:
        slots[2] = -1                                   # padding: rotated, not cached
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    before = f64(kp), f64(vp)
    ins = [f64(x) for x in (q, k, v)]
    out = binding.rope_append(q if Hq else None, k, v, pos, inv, slots, kp, vp, interleaved=interleaved,
                              mscale=1.5, dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    p, iv = pos.cpu().numpy(), inv.cpu().numpy().astype(np.float64)
    if Hq:
        check_values(out, oracle.rope(ins[0], p, iv, interleaved, 1.5),
                     rotated_bound(ins[0], rd, interleaved, 1.5, dtype), dtype)
        assert torch.equal(out[..., rd:], q[..., rd:])
    else:
        assert out is None
    kw, tol = before[0], np.zeros_like(before[0])
    oracle.kv_append(kw, before[1], oracle.rope(ins[1], p, iv, interleaved, 1.5), ins[2], slots.cpu().numpy())
    oracle.kv_append(tol, np.zeros_like(tol), rotated_bound(ins[1], rd, interleaved, 1.5, dtype),
                     ins[2], slots.cpu().numpy())
    check_values(kp, kw, tol + (np.abs(kw) * 0), dtype)
    assert np.array_equal(f64(vp), before[1])            # values are copied bit for bit


def test_unwritten_rows_keep_their_bits_and_inputs_stay():
    q, k, v, pos, slots, kp, vp = make(3, 20, 4, 2, 128, 16, torch.bfloat16, 5000, True)
    slots[::3] = -1
    mine = torch.zeros(kp.shape[0] * 16, dtype=torch.bool, device="cuda")
    mine[slots[slots >= 0]] = True
    before, qkv = kp.clone(), q.clone()
    inv, m = binding.rope_frequencies(128)
    binding.rope_append(q, k, v, pos, inv, slots, kp, vp, mscale=m)
    rows = kp.transpose(1, 2).reshape(-1, 2, 128)
    old = before.transpose(1, 2).reshape(-1, 2, 128)
    assert torch.equal(rows[~mine], old[~mine]) and torch.equal(q, qkv)


def test_rotates_q_in_place():
    q, k, v, pos, slots, kp, vp = make(4, 33, 8, 2, 64, 16, torch.bfloat16, 9000, False)
    inv, m = binding.rope_frequencies(64, scaling="yarn", factor=8.0)
    want = binding.rope_append(q, k, v, pos, inv, slots, kp, vp, mscale=m)
    got = binding.rope_append(q, k, v, pos, inv, slots, kp, vp, mscale=m, q_out=q)
    assert got.data_ptr() == q.data_ptr() and torch.equal(got, want)


def test_slots_past_the_pool_are_reported_and_skipped():
    q, k, v, pos, slots, kp, vp = make(5, 8, 2, 1, 64, 16, torch.float32, 100, False)
    slots[3] = kp.shape[0] * 16
    slots[5] = 1 << 40
    inv, _ = binding.rope_frequencies(64)
    guard = kp.clone()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    binding.rope_append(q, k, v, pos, inv, slots, kp, vp, dev_err=err)
    assert int(err.item()) == binding.DEVERR_SLOT
    assert (kp != guard).any(-1).sum() == 6


@pytest.mark.parametrize("D,rd,bs", [(64, 64, 16), (128, 96, 32), (256, 256, 16)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_q4_quantises_the_rotated_rows(D, rd, bs, interleaved):
    """Into 4-bit pools: exactly what kv_append_q4 writes of the rotated,
    rounded keys (which the 16-bit call gives)."""
    T, Hq, Hkv = 45, 4, 2
    q, k, v, pos, slots, kp, vp = make(D, T, Hq, Hkv, D, bs, torch.bfloat16, 70000, True)
    slots[7] = -1
    inv, m = binding.rope_frequencies(rd, scaling="ntk", factor=4.0)
    want_q = binding.rope_append(q, k, v, pos, inv, slots, kp, vp, interleaved=interleaved, mscale=m)
    k4, v4 = binding.q4_pools(kp.shape[0], Hkv, bs, D)
    k4.random_()
    v4.random_()
    wk, wv = k4.clone(), v4.clone()
    got_q = binding.rope_append(q, k, v, pos, inv, slots, k4, v4, interleaved=interleaved, mscale=m)
    assert torch.equal(got_q, want_q)
    rows = kp.transpose(1, 2).reshape(-1, Hkv, D)[slots.clamp(min=0)].contiguous()
    binding.kv_append_q4(rows, v, slots, wk, wv)
    assert torch.equal(k4, wk) and torch.equal(v4, wv)


@pytest.mark.parametrize("fused", [False, True])
def test_other_stream_and_graph(fused):
    q, k, v, pos, slots, kp, vp = make(6, 50, 4, 2, 128, 16, torch.bfloat16, 4000, fused)
    inv, m = binding.rope_frequencies(128, scaling="linear", factor=2.0)
    want = binding.rope_append(q, k, v, pos, inv, slots, kp, vp, mscale=m)
    kw = kp.clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    kp.zero_()
    torch.cuda.synchronize()
    out = torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        binding.rope_append(q, k, v, pos, inv, slots, kp, vp, mscale=m, q_out=out)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    rows, old = (x.transpose(1, 2).reshape(-1, 2, 128)[slots] for x in (kp, kw))
    assert torch.equal(rows, old)
