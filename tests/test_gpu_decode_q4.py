"""pa_decode_q4 against the 64-bit definition on the values that the pools stand
for.

Bound of an output element, with w_t the softmax weights, v = mid + s (c - 8):
* p s is rounded to bf16, half a step of 2^-8: 2^-8 sum w s |c - 8|;
* the output is rounded to bf16: 2^-8 |out|;
* a logit's group sum starts at -128 Q and takes four products of codes up to
  143 with q in fp32 accumulators, each off by at most a step (2^-23) of what
  passes through them, less than 271 sum |q|: e = scale s 4 * 2^-23 * 271
  sum |q|, doubled for the products' inner sums; a logit off by e moves an
  output by at most 2 e sum w |v|;
* exp2, the fp32 sums and the start value of O (which cancels at most 64 tokens
  of 136 s p, against sum w s |c - 8|): 2^-18 of sum w (|v| + 16 s)."""

import numpy as np
import pytest
import torch

import oracle
from oracle import serving_ops as so
from paged_kv_cache_336_b200 import binding

pytestmark = pytest.mark.gpu


def make(seed, lens, Hq, Hkv, D, bs, s_lo=0.1, s_hi=0.5, slack=1):
    """Random 4-bit pools (scales up to s_hi, minima near -8 scales), shuffled tables."""
    rng = np.random.default_rng(seed)
    B, mbs = len(lens), max(1, max(-(-n // bs) for n in lens)) + slack
    nb = sum(-(-n // bs) for n in lens) + 5
    ids = rng.permutation(nb)
    tables = np.full((B, mbs), -1, dtype=np.int32)
    k = 0
    for s, n in enumerate(lens):
        for i in range(-(-n // bs)):
            tables[s, i] = ids[k]
            k += 1
    pools = []
    for _ in range(2):
        pool = rng.integers(0, 256, (nb, Hkv, bs // 16, 9 * D), dtype=np.uint8)
        sc = rng.uniform(s_lo, s_hi, (nb, Hkv, bs // 16, 16, D // 64))
        mn = -7.5 * sc + rng.standard_normal(sc.shape) * s_hi
        bits = np.stack([so.bf16_bits(sc), so.bf16_bits(mn)], -1)
        pool[..., 8 * D:] = bits.reshape(*bits.shape[:3], -1).view(np.uint8)
        pools.append(pool.reshape(nb, Hkv, -1))
    q = torch.from_numpy(rng.standard_normal((B, Hq, D))).to(torch.bfloat16)
    return q, pools[0], pools[1], tables, np.asarray(lens, dtype=np.int32)


def dense(pool, D, bs, value):
    """(values, s (c - 8), s) of a pool as [NB, Hkv, bs, D]."""
    NB, H = pool.shape[:2]
    sub = pool.reshape(NB, H, bs // 16, 9 * D)
    codes = sub[..., :8 * D].reshape(NB, H, bs // 16, 16, D // 2)
    nib = np.stack([codes & 15, codes >> 4], -1).reshape(NB, H, bs // 16, 16, D).astype(np.float64)
    at = np.empty((16, D), dtype=np.int64)
    for r in range(16):
        for c in range(D // 8):
            at[r, 8 * c:8 * c + 8] = 2 * so.q4_word_offset(r, c, D, value) + np.arange(8)
    code = np.take_along_axis(nib, np.broadcast_to(at, nib.shape), -1)
    pair = so.bf16_value(np.ascontiguousarray(sub[..., 8 * D:]).view(np.uint16))
    pair = pair.reshape(NB, H, bs // 16, 16, D // 64, 2).astype(np.float64).repeat(64, -2)
    flat = [x.reshape(NB, H, bs, D) for x in
            (pair[..., 1] + pair[..., 0] * code, pair[..., 0] * (code - 8), pair[..., 0])]
    return flat


def test_dense_helper_is_the_oracles():
    q, k, v, _, _ = make(1, [20], 1, 2, 128, 32)
    for pool, value in ((k, False), (v, True)):
        assert np.array_equal(dense(pool, 128, 32, value)[0], oracle.q4_dense(pool, 128, 32, value))


def check(q, kp, vp, tables, lens, bs, window=0, sinks=0, partition_tokens=64, scale=None, out=None):
    B, Hq, D = q.shape
    scale = 1 / np.sqrt(D) if scale is None else scale
    kd, _, ks = dense(kp, D, bs, False)
    vd, vc, vs = dense(vp, D, bs, True)
    q64 = q.double().numpy()

    def attend(values):
        return oracle.paged_decode_sinks(q64, kd, values, tables, lens, scale, window, sinks)

    want = attend(vd)
    # broadcast a bound on the logits over heads: scale * s * sum |q| per query head
    e = 2 * abs(scale) * ks.max() * 4 * 2.0 ** -23 * 271 * np.abs(q64).sum(-1, keepdims=True)
    tol = 2.0 ** -8 * (attend(np.abs(vc)) + np.abs(want)) + 2 * e * attend(np.abs(vd)) + \
        2.0 ** -18 * attend(np.abs(vd) + 16 * vs)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = binding.decode_q4(q.cuda(), torch.from_numpy(kp).cuda(), torch.from_numpy(vp).cuda(),
                            torch.from_numpy(tables).cuda(), torch.from_numpy(lens).cuda(), scale,
                            window=window, sinks=sinks, partition_tokens=partition_tokens, dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    g = got.double().cpu().numpy()
    assert np.all(np.isfinite(g))
    bad = np.abs(g - want) - tol
    assert np.all(bad <= 0), (float(bad.max()), np.unravel_index(bad.argmax(), bad.shape))
    return got


LENS = [0, 1, 15, 16, 17, 63, 64, 65, 200, 129]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("bs", [16, 32])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 2), (8, 1), (12, 2), (16, 1), (18, 2)])
def test_matches_definition(D, bs, Hq, Hkv):
    check(*make(D + bs + Hq, LENS, Hq, Hkv, D, bs), bs)


@pytest.mark.parametrize("D,bs", [(64, 32), (128, 16), (256, 16)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (17, 4), (40, 0), (64, 16), (70, 37), (33, 150),
                                          (5000, 4)])
def test_windows_and_sinks(D, bs, window, sinks):
    q, k, v, tables, lens = make(window + sinks, LENS, 8, 2, D, bs)
    hidden = tables.copy()                # blocks without a visible token are released
    if window:
        for s, n in enumerate(lens):
            for b in range(tables.shape[1]):
                t = np.arange(b * bs, min((b + 1) * bs, n))
                if not ((t >= n - window) | (t < sinks)).any():
                    hidden[s, b] = -1
    check(q, k, v, hidden, lens, bs, window, sinks)


@pytest.mark.parametrize("partition_tokens", [32, 512])
def test_many_pieces(partition_tokens):
    check(*make(5, [5000, 17, 2999, 0, 1024], 8, 2, 128, 16), 16, partition_tokens=partition_tokens)


def test_one_long_sequence():
    check(*make(6, [20001], 4, 1, 128, 16), 16, partition_tokens=512)


def test_many_short_sequences():
    rng = np.random.default_rng(8)
    lens = rng.integers(0, 40, 700).tolist()
    check(*make(7, lens, 2, 1, 64, 16), 16)


def test_negative_scale_and_tiny_and_large_steps():
    check(*make(9, LENS, 4, 2, 128, 16), 16, scale=-0.2)
    check(*make(10, LENS, 4, 2, 128, 16, s_lo=1e-20, s_hi=1e-19), 16)
    q, k, v, tables, lens = make(11, LENS, 4, 2, 64, 16, s_lo=2.0 ** 60, s_hi=2.0 ** 61)
    check(q, k, v, tables, lens, 16, scale=2.0 ** -64)


def test_rows_that_are_not_visible_may_hold_anything():
    """All-ones bytes (codes 15, scale and minimum NaN) wherever nothing is visible."""
    bs, D, window, sinks = 32, 128, 21, 5
    q, k, v, tables, lens = make(12, [200, 31, 22, 1, 100], 8, 2, D, bs)
    want = check(q, k, v, tables, lens, bs, window, sinks)
    see = np.zeros((k.shape[0], bs), dtype=bool)
    for s, n in enumerate(lens):
        for t in range(n):
            if t >= n - window or t < sinks:
                see[tables[s, t // bs], t % bs] = True
    for pool in (k, v):
        sub = pool.reshape(pool.shape[0], 2, bs // 16, 9 * D)
        for b in range(pool.shape[0]):
            for t in range(bs):
                if not see[b, t]:
                    r = t % 16
                    sub[b, :, t // 16, r * D // 2:(r + 1) * D // 2] = 0xff
                    sub[b, :, t // 16, 8 * D + r * D // 16:8 * D + (r + 1) * D // 16] = 0xff
    got = binding.decode_q4(q.cuda(), torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(),
                            torch.from_numpy(tables).cuda(), torch.from_numpy(lens).cuda(),
                            1 / np.sqrt(D), window=window, sinks=sinks, partition_tokens=64)
    assert torch.equal(got, want)


def test_a_nan_that_is_visible_reaches_the_output():
    q, k, v, tables, lens = make(13, [40, 40], 2, 1, 64, 16)
    at = v.reshape(v.shape[0], 1, 9 * 64)[tables[0, 1], 0]
    at[512 + 4 * 3:512 + 4 * 3 + 4] = 0xff
    args = [torch.from_numpy(x).cuda() for x in (k, v, tables, lens)]
    got = binding.decode_q4(q.cuda(), *args, 0.1)
    assert torch.isnan(got[0]).all() and torch.isfinite(got[1]).all()


def test_bad_blocks_and_lengths_are_reported():
    q, k, v, tables, lens = make(14, [40, 50, 20], 4, 2, 64, 16)
    args = [torch.from_numpy(x).cuda() for x in (k, v, tables, lens)]
    want = binding.decode_q4(q.cuda(), *args, 0.1)
    tables[0, 1] = k.shape[0]
    lens[2] = 16 * tables.shape[1] + 1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = [torch.from_numpy(x).cuda() for x in (k, v, tables, lens)]
    got = binding.decode_q4(q.cuda(), *args, 0.1, dev_err=err)
    assert int(err.item()) == binding.DEVERR_BLOCK_ID | binding.DEVERR_CONTEXT_LEN
    assert torch.equal(got[1], want[1]) and torch.all(got[2] == 0)
    assert not torch.equal(got[0], want[0]) and torch.isfinite(got[0]).all()


def test_workspace_is_reused_and_results_repeat():
    """Bit-equal results from one workspace over different batches, from a
    captured graph, and with a dirty workspace."""
    q, k, v, tables, lens = make(15, [3000, 17, 0, 500], 8, 2, 128, 16)
    args = [torch.from_numpy(x).cuda() for x in (k, v, tables, lens)]
    q = q.cuda()
    ws = binding.SplitWorkspace(4, 8, 128, 16, tables.shape[1], 64)
    a = binding.decode_q4(q, *args, 0.1, workspace=ws)
    binding.decode_q4(q, *args, 0.3, window=30, sinks=3, workspace=ws)
    ws.buffer[512:].fill_(0xff)
    b = binding.decode_q4(q, *args, 0.1, workspace=ws)
    assert torch.equal(a, b)
    out = torch.empty_like(a)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        binding.decode_q4(q, *args, 0.1, workspace=ws, out=out)
    for _ in range(3):
        out.zero_()
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, a)


def test_a_long_sequence_of_bad_blocks_gives_zeros():
    """Every block id outside the pool, the work cut into many pieces: zeros and
    the error bit, beside an untouched neighbour."""
    q, k, v, tables, lens = make(16, [3000, 40], 4, 2, 64, 16)
    args = [torch.from_numpy(x).cuda() for x in (k, v, tables, lens)]
    want = binding.decode_q4(q.cuda(), *args, 0.1, partition_tokens=32)
    args[2][0] = 10 ** 6
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = binding.decode_q4(q.cuda(), *args, 0.1, partition_tokens=32, dev_err=err)
    assert int(err.item()) == binding.DEVERR_BLOCK_ID
    assert torch.all(got[0] == 0) and torch.equal(got[1], want[1])


def test_the_most_sequences():
    rng = np.random.default_rng(17)
    lens = rng.integers(0, 20, 4096).tolist()
    check(*make(17, lens, 1, 1, 64, 16), 16)


def test_scales_that_grow_and_a_nan_beside_them():
    """Value scales over 2^-30 .. 2^30, rising along the sequence; then a NaN
    scale in one group, which leaves the other group's dims as they were."""
    q, k, v, tables, lens = make(18, [333, 200], 4, 1, 128, 16)
    sub = v.reshape(v.shape[0], 1, 9 * 128)
    for s in range(2):
        for b in range(-(-int(lens[s]) // 16)):
            par = np.ascontiguousarray(sub[tables[s, b], 0, 1024:]).view(np.uint16).reshape(16, 2, 2)
            val = so.bf16_value(par) * 2.0 ** (-30 + 60 * b / 21)
            sub[tables[s, b], 0, 1024:] = so.bf16_bits(val).reshape(-1).view(np.uint8)
    want = check(q, k, v, tables, lens, 16, scale=0.02)
    sub[tables[0, 3], 0, 1024 + 8 * 5:1024 + 8 * 5 + 4] = 0xff       # token 53, dims 0 .. 63
    args = [torch.from_numpy(x).cuda() for x in (k, v, tables, lens)]
    got = binding.decode_q4(q.cuda(), *args, 0.02, partition_tokens=64)
    assert torch.isnan(got[0, :, :64]).all() and torch.equal(got[0, :, 64:], want[0, :, 64:])
    assert torch.equal(got[1], want[1])


def test_offsets_past_32_bits():
    """Pools of more than 4 GiB, sequences in their last blocks: append, read
    back, attention, and rope_append into 16-bit pools of that size."""
    D, H, bs = 256, 8, 32
    NB = (1 << 32) // (H * 9 * D * 2) + 200
    kp, vp = (torch.empty(NB, H, 2 * 9 * D, dtype=torch.uint8, device="cuda") for _ in range(2))
    T = 100
    g = torch.Generator(device="cuda").manual_seed(19)
    k, v = (torch.randn(T, H, D, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    q = torch.randn(1, H, D, device="cuda", generator=g).to(torch.bfloat16)
    blocks = torch.arange(NB - 1, NB - 5, -1, device="cuda")
    slots = (blocks[:, None] * bs + torch.arange(bs, device="cuda")).flatten()[:T]
    binding.kv_append_q4(k, v, slots, kp, vp)
    small = [torch.empty(4, H, 2 * 9 * D, dtype=torch.uint8, device="cuda") for _ in range(2)]
    near = torch.arange(T, device="cuda")
    binding.kv_append_q4(k, v, near, *small)
    for a, b in zip(binding.kv_gather_q4(kp, vp, slots, D), binding.kv_gather_q4(*small, near, D)):
        assert torch.equal(a, b)
    ctx = torch.tensor([T], dtype=torch.int32, device="cuda")
    a = binding.decode_q4(q, kp, vp, blocks.to(torch.int32)[None], ctx, 0.06)
    b = binding.decode_q4(q, *small, torch.arange(4, dtype=torch.int32, device="cuda")[None], ctx, 0.06)
    assert torch.equal(a, b)
    del kp, vp
    NB = (1 << 32) // (H * bs * D * 2) + 100
    kp = torch.empty(NB, H, bs, D, dtype=torch.bfloat16, device="cuda")
    vp = torch.empty_like(kp)
    slots = torch.arange(NB * bs - T, NB * bs, device="cuda")
    inv, m = binding.rope_frequencies(D)
    binding.rope_append(None, k, v, torch.zeros(T, dtype=torch.int32, device="cuda"), inv, slots, kp, vp, mscale=m)
    rows = vp[-4:].transpose(1, 2).reshape(-1, H, D)[-T:]
    assert torch.equal(rows, v)
    rows = kp[-4:].transpose(1, 2).reshape(-1, H, D)[-T:]
    assert torch.equal(rows, k)                       # position 0: nothing turns


@pytest.mark.parametrize("num,Hkv", [(1, 1), (7, 5), (300, 2), (1200, 3)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (30, 3)])
def test_short_sequences_whole_and_cut(num, Hkv, window, sinks):
    """Sequences of at most eight units: one warp each while a wave of CTAs holds
    them, an equal cut beyond."""
    rng = np.random.default_rng(num)
    lens = [127, 0][:num] + rng.integers(0, 128, max(0, num - 2)).tolist()
    check(*make(num, lens, 2 * Hkv, Hkv, 128, 16, slack=0), 16, window, sinks)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("top", [63, 100, 190, 380, 700])
def test_every_number_of_pieces_in_a_cta(D, top):
    """One sequence of `top` tokens sets how many warps share each sequence; the
    others leave some of them without units. Nine query heads: two runs of heads."""
    check(*make(D + top, [top, 1, 0, top // 2, 17], 18, 2, D, 16, slack=0), 16, partition_tokens=512)


def test_pieces_in_a_cta_equal_equal_runs():
    """The same sequences in a small batch (merged in the CTA) and in a batch that a
    wave cannot hold (equal runs and the merge kernel)."""
    q, k, v, tables, lens = make(23, [300, 1, 160] + [200] * 900, 4, 2, 64, 16, slack=0)
    args = [torch.from_numpy(x).cuda() for x in (k, v, tables, lens)]
    many = binding.decode_q4(q.cuda(), *args, 0.1)
    few = binding.decode_q4(q[:3].cuda(), *args[:2], args[2][:3].contiguous(), args[3][:3], 0.1)
    # both within the bound of check(); against each other twice that, here two bf16 steps
    assert torch.all((many[:3].float() - few.float()).abs() <= 2.0 ** -6 * few.float().abs() + 2e-2)
    check(q[:3], k, v, tables[:3], lens[:3], 16)


@pytest.mark.parametrize("D,num,window,sinks", [(64, 420, 0, 0), (64, 420, 131, 5), (256, 140, 0, 0), (256, 140, 50, 3)])
def test_whole_steps_and_their_remainders(D, num, window, sinks):
    """Runs of many steps for every warp: sequences around whole steps (eight units
    at head_dim 64, three at 256) and such that end inside one."""
    rng = np.random.default_rng(D + window)
    lens = [127, 128, 129, 255, 256, 257, 47, 48, 49, 95, 96, 97] + rng.integers(100, 330, num - 12).tolist()
    check(*make(D, lens, 16, 8, D, 16 if window else 32, slack=0), 16 if window else 32, window, sinks)
