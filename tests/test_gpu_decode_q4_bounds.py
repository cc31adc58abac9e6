"""pa_decode_q4 against the 64-bit definition, within a bound derived from the
arithmetic that include/pagedkv.h states, over value scales and minima that lie
far apart and in every way in which a batch is cut.

Notation: a visible token t has key k = mn + s c and value v = mn + s c (each
with its own s, mn and codes c), logit z = scale q.k, weight w = softmax(z);
L = sum exp(z - max z) >= 1; n tokens.

* q enters as rint(2^k q), its head's largest |q| brought to 2^14 or more, so
  each is off by at most 2^-15 max|q|. It meets the codes only (the minima
  meet the sum of q itself): a logit is off by 2^-15 max|q| |scale| sum_d s c.
* The code products are exact. Everything else of a logit is fp32: the sum of
  64 q (18 additions in a row), one conversion, two operations for each of at
  most four groups, the scaling and the subtraction of the maximum: below 2^5
  roundings of 2^-24 of |scale| sum_d (s c + |mn|) |q|.
  Together E, taken at the token where it is largest. Logits off by E move
  each weight by a factor within exp(+-2 E), the output by at most
  (exp(2 E) - 1) sum w |v|.
* exp2 and the factors that join pieces: 2^-19 sum w |v|.
* A weight times the value's scale becomes f16: 2^-11 of it, and where it falls
  below f16's normal numbers 2^-39 of the group's largest scale times the
  largest weight so far: sum w s |c - 8| 2^-11 + 8 n 2^-39 max s / L.
* O and the minima's sum are fp32 sums, over at most n / 16 + 32 steps (n / 8
  additions for the minima): (n / 8 + 32) 2^-23 sum w (s |c - 8| + |mn + 8 s|).
* The output is rounded to bf16: 2^-8 of it."""

import numpy as np
import pytest
import torch

from oracle import serving_ops as so
from paged_kv_cache_336_b200 import binding

from test_gpu_decode_q4 import make

gpu = pytest.mark.gpu


def fields(pool, D, bs, value):
    """(s, mn, c) of a pool, each [NB, Hkv, bs, D] in 64 bits."""
    NB, H = pool.shape[:2]
    sub = pool.reshape(NB, H, bs // 16, 9 * D)
    rows = sub[..., :8 * D].reshape(NB, H, bs // 16, 16, D // 2)
    nib = np.stack([rows & 15, rows >> 4], -1).reshape(NB, H, bs // 16, 16, D).astype(np.float64)
    at = np.array([[2 * so.q4_word_offset(r, d // 8, D, value) + d % 8 for d in range(D)] for r in range(16)])
    code = np.take_along_axis(nib, np.broadcast_to(at, nib.shape), -1)
    pair = so.bf16_value(np.ascontiguousarray(sub[..., 8 * D:]).view(np.uint16)).astype(np.float64)
    pair = pair.reshape(NB, H, bs // 16, 16, D // 64, 2).repeat(64, -2)
    return [x.reshape(NB, H, bs, D) for x in (pair[..., 0], pair[..., 1], code)]


def definition(q, K, V, scale):
    """(output, bound) of one query row over visible tokens; K, V: (s, mn, c), [n, D]."""
    (ks, km, kc), (vs, vm, vc) = K, V
    n = len(ks)
    z = scale * ((km + ks * kc) @ q)
    E = abs(scale) * (2.0 ** -15 * np.abs(q).max() * (ks * kc).sum(-1) +
                      2.0 ** -19 * ((ks * kc + np.abs(km)) @ np.abs(q)))
    e = np.exp(z - z.max())
    w, L = e / e.sum(), e.sum()
    v = vm + vs * vc
    out = w @ v
    moved = (np.expm1(2 * E.max()) + 2.0 ** -19) * (w @ np.abs(v))
    weights = 2.0 ** -11 * (w @ (vs * np.abs(vc - 8))) + 8 * n * 2.0 ** -39 * vs.max(0) / L
    sums = (n / 8 + 32) * 2.0 ** -23 * (w @ (vs * np.abs(vc - 8) + np.abs(vm + 8 * vs)))
    return out, 2.0 ** -8 * np.abs(out) + (1 + 2.0 ** -8) * (moved + weights + sums)


def visible(n, window, sinks):
    t = np.arange(n)
    return t if not window else t[(t >= n - window) | (t < sinks)]


def check_rows(got, q, kp, vp, tables, lens, bs, window=0, sinks=0, scale=0.1):
    """Every row of the first len(lens) sequences against the bound."""
    D = q.shape[-1]
    K, V = fields(kp, D, bs, False), fields(vp, D, bs, True)
    q64, g = q.double().cpu().numpy(), got.double().cpu().numpy()
    assert np.all(np.isfinite(g))
    group = q.shape[1] // kp.shape[1]
    worst = 0.0
    for s, n in enumerate(lens):
        if n == 0:
            assert np.all(g[s] == 0)
            continue
        t = visible(int(n), window, sinks)
        b = tables[s][t // bs]
        for h in range(q.shape[1]):
            want, tol = definition(q64[s, h], [x[b, h // group, t % bs] for x in K],
                                   [x[b, h // group, t % bs] for x in V], scale)
            off = np.abs(g[s, h] - want)
            assert np.all(off <= tol), (s, h, float((off - tol).max()), int((off - tol).argmax()))
            worst = max(worst, float((off / tol).max()))
    return worst


def run(q, kp, vp, tables, lens, **kw):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = binding.decode_q4(q.cuda(), torch.from_numpy(kp).cuda(), torch.from_numpy(vp).cuda(),
                            torch.from_numpy(tables).cuda(), torch.from_numpy(lens).cuda(), kw.pop("scale", 0.1),
                            dev_err=err, **kw)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    return out


def many(q, tables, lens, lists):
    """The batch followed by copies of its longest sequence, beyond what one wave of
    warps holds."""
    count = 2 * torch.cuda.get_device_properties(0).multi_processor_count * 12 // lists + 64
    at = int(np.argmax(lens))
    assert len(lens) + count <= 4096
    return (torch.cat([q, q[at:at + 1].expand(count, -1, -1)]).contiguous(),
            np.concatenate([tables, np.repeat(tables[at:at + 1], count, 0)]),
            np.concatenate([lens, np.full(count, lens[at], dtype=np.int32)]))


def both_ways(q, kp, vp, tables, lens, bs, window=0, sinks=0, scale=0.1):
    """The batch alone (pieces merged in a CTA) and inside a large one (equal runs)."""
    few = run(q, kp, vp, tables, lens, window=window, sinks=sinks, scale=scale, partition_tokens=512)
    check_rows(few, q, kp, vp, tables, lens, bs, window, sinks, scale)
    lists = kp.shape[1] * -(-(q.shape[1] // kp.shape[1]) // 8)
    q2, tables2, lens2 = many(q, tables, lens, lists)
    out = run(q2, kp, vp, tables2, lens2, window=window, sinks=sinks, scale=scale, partition_tokens=32)
    check_rows(out, q, kp, vp, tables, lens, bs, window, sinks, scale)
    at = int(np.argmax(lens))
    assert torch.isfinite(out).all()
    check_rows(out[-1:], q[at:at + 1], kp, vp, tables[at:at + 1], lens[at:at + 1], bs, window, sinks, scale)


LENS = [300, 1, 16, 0, 177, 48, 64, 129]


@gpu
@pytest.mark.parametrize("D,bs,Hq,Hkv", [(64, 16, 4, 2), (128, 32, 8, 1), (128, 16, 20, 2), (256, 16, 2, 1)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 5)])
def test_within_the_bound(D, bs, Hq, Hkv, window, sinks):
    both_ways(*make(D + Hq, LENS, Hq, Hkv, D, bs, slack=0), bs, window, sinks)


@gpu
def test_a_query_with_one_dim_far_above_the_rest():
    q, kp, vp, tables, lens = make(3, LENS, 4, 2, 128, 16, slack=0)
    q[..., 7] *= 1000
    both_ways(q, kp, vp, tables, lens, 16, scale=0.002)


def set_values(vp, D, bs, s, mn):
    """Value parameters: s, mn broadcast to [NB, Hkv, tokens of a block, D / 64]."""
    sub = vp.reshape(vp.shape[0], vp.shape[1], bs // 16, 9 * D)
    shape = (*sub.shape[:3], 16, D // 64)
    pair = [so.bf16_bits(np.broadcast_to(np.asarray(x, dtype=np.float64), shape)) for x in (s, mn)]
    sub[..., 8 * D:] = np.stack(pair, -1).reshape(*sub.shape[:3], -1).view(np.uint8)


@gpu
@pytest.mark.parametrize("D,powers", [(128, (0, -30)), (128, (0, -45)), (128, (-100, 3)), (128, (90, -110)),
                                      (256, (0, -40, 30, -80)), (256, (-60, -60, 60, 0)), (64, (-110,)), (64, (95,))])
def test_groups_of_scales_far_apart(D, powers):
    """Each 64-dim group keeps its own bits, however large the scales beside it."""
    q, kp, vp, tables, lens = make(abs(sum(powers)), LENS, 4, 2, D, 16, slack=0)
    rng = np.random.default_rng(5)
    s = 2.0 ** np.asarray(powers, dtype=np.float64) * rng.uniform(0.5, 1, (vp.shape[0], 2, 1, 16, D // 64))
    set_values(vp, D, 16, s, -7.3 * s)
    both_ways(q, kp, vp, tables, lens, 16)


@gpu
@pytest.mark.parametrize("power", [0, 60, 96])
@pytest.mark.parametrize("s", [0.0, 2.0 ** -60, 1.0])
def test_minima_far_above_the_scales(power, s):
    """Flat groups (scale 0) and such whose scale is nothing beside the minimum."""
    q, kp, vp, tables, lens = make(power, [5000, 700, 16, 1], 4, 1, 64, 16, slack=0)
    rng = np.random.default_rng(6)
    set_values(vp, 64, 16, s, 2.0 ** power * rng.uniform(0.5, 1, (vp.shape[0], 1, 1, 16, 1)))
    both_ways(q, kp, vp, tables, lens, 16, scale=0.001)


@gpu
@pytest.mark.parametrize("low,high", [(-110, 90), (90, -110)])
def test_scales_that_change_along_the_sequence(low, high):
    q, kp, vp, tables, lens = make(8, [333, 200, 40], 4, 1, 128, 16, slack=0)
    sub = np.zeros((vp.shape[0], 1, 1, 16, 2))
    for i, n in enumerate(lens):
        for b in range(-(-int(n) // 16)):
            sub[tables[i, b]] = 2.0 ** (low + (high - low) * b / 21)
    set_values(vp, 128, 16, sub, -6 * sub)
    both_ways(q, kp, vp, tables, lens, 16, scale=0.02)


# ---------------------------------------------------------------------------
# A case whose outputs nearly cancel, so that neither their rounding nor the
# logits' hides that of the weights.

def cancelling(num=64, Hq=8, D=64, bs=16):
    """Sequences of two tokens. Keys are flat (s = 0), so the logits are scale mn sum q
    and q's rounding does not enter; values x s_A and -x s_B with minima -8 s, and
    s_B the bf16 number next to w_A s_A / w_B for head 0 (the other heads hold the
    same query)."""
    rng = np.random.default_rng(11)
    q = torch.from_numpy(rng.standard_normal((num, 1, D))).to(torch.bfloat16).expand(num, Hq, D).contiguous()
    kp = np.zeros((num, 1, 9 * D), dtype=np.uint8)
    vp = np.zeros_like(kp)
    tables = np.arange(num, dtype=np.int32)[:, None].copy()
    lens = np.full(num, 2, dtype=np.int32)
    total = q[:, 0].double().sum(-1).numpy()
    for s in range(num):
        gap = rng.uniform(0.1, 1.5) / (0.1 * total[s])     # z_A - z_B near 0.1 .. 1.5
        km = so.bf16_value(so.bf16_bits(np.array([gap, 0.0]))).astype(np.float64)
        z = 0.1 * km * total[s]
        w = np.exp(z - z.max()) / np.exp(z - z.max()).sum()
        sa = rng.uniform(0.5, 1)
        sv = so.bf16_value(so.bf16_bits(np.array([sa, 0.0]))).astype(np.float64)
        sv[1] = so.bf16_value(so.bf16_bits(np.array([w[0] * sv[0] / w[1]])))[0]
        x = rng.integers(-7, 8, D)
        for t in range(2):
            at = 8 * D + 4 * t
            kp[s, 0, at:at + 4] = np.array([so.bf16_bits(0.0), so.bf16_bits(km[t])], dtype=np.uint16).view(np.uint8)
            vp[s, 0, at:at + 4] = np.array([so.bf16_bits(sv[t]), so.bf16_bits(-8 * sv[t])], dtype=np.uint16).view(np.uint8)
            for c in range(D // 8):
                codes = 8 + (x if t == 0 else -x)[8 * c:8 * c + 8]
                word = sum(int(v) << (4 * j) for j, v in enumerate(codes))
                off = t * D // 2 + so.q4_word_offset(t, c, D, True)
                vp[s, 0, off:off + 4] = np.frombuffer(np.uint32(word).tobytes(), dtype=np.uint8)
    return q, kp, vp, tables, lens


def rounded_weights(q, kp, vp, tables, lens, dtype, scale=0.1):
    """What the call would give with weights times scales rounded to `dtype`."""
    D = q.shape[-1]
    (_, km, _), (vs, vm, vc) = fields(kp, D, 16, False), fields(vp, D, 16, True)
    out = torch.empty(q.shape, dtype=torch.bfloat16)
    for s in range(len(lens)):
        z = scale * km[s, 0, :2, 0] * q[s, 0].double().sum().item()
        e = np.exp(z - z.max())
        ps = torch.from_numpy(e[:, None] * vs[s, 0, :2]).to(dtype).double().numpy()
        o = (ps * (vc[s, 0, :2] - 8)).sum(0) + (e[:, None] * (vm + 8 * vs)[s, 0, :2]).sum(0)
        out[s] = torch.from_numpy(o / e.sum()).to(torch.bfloat16)
    return out


def test_the_bound_tells_16_bit_weights_apart():
    """On the oracle alone: weights rounded to f16 pass, weights rounded to bf16 do not."""
    case = cancelling()
    assert check_rows(rounded_weights(*case, torch.float16), *case, 16) <= 1
    with pytest.raises(AssertionError):
        check_rows(rounded_weights(*case, torch.bfloat16), *case, 16)


@gpu
def test_outputs_that_nearly_cancel():
    case = cancelling()
    check_rows(run(*case), *case, 16)
