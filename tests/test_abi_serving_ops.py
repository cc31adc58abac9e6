"""CPU tests of the serving-step entry points: refusals before the device is
touched, sizes and frequencies computed on the host, and the Python layer's
own checks (on CPU tensors, which it refuses before any call)."""

import ctypes
import math

import numpy as np
import pytest
import torch

from paged_kv_cache_336_b200 import binding
from paged_kv_cache_336_b200.binding import InvalidArgumentError, PagedKVError

FAKE = 0x7000_0000  # aligned host address never dereferenced: validation fails first
BAD, UNSUP, OK = binding.PA_ERR_INVALID_ARG, binding.PA_ERR_UNSUPPORTED, binding.PA_OK
BF16, F32 = binding.PA_BF16, binding.PA_F32


def call(name, defaults, over, order):
    a = {**defaults, **over}
    return getattr(binding.library(), name)(*[a[k] for k in order])


DECODE = dict(q=FAKE, k=FAKE, v=FAKE, bt=FAKE, ctx=FAKE, B=4, Hq=8, Hkv=2, D=128, BS=16, NB=64, MBS=8,
              scale=0.1, dtype=BF16, window=32, sinks=4, pt=64, ws=FAKE, wsb=1 << 40, out=FAKE, err=None,
              stream=None)
SINKS_ORDER = "q k v bt ctx B Hq Hkv D BS NB MBS scale dtype pt window sinks ws wsb out err stream".split()
Q4_ORDER = "q k v bt ctx B Hq Hkv D BS NB MBS scale dtype window sinks pt ws wsb out err stream".split()

COMMON = [
    (dict(q=None), BAD), (dict(bt=None), BAD), (dict(out=FAKE + 8), BAD), (dict(k=FAKE + 4), BAD),
    (dict(Hq=7), BAD), (dict(NB=0), BAD), (dict(scale=float("inf")), BAD), (dict(dtype=5), BAD),
    (dict(B=-1), BAD), (dict(sinks=-1), BAD), (dict(pt=24), BAD), (dict(pt=0), BAD), (dict(ws=None), BAD),
    (dict(ws=FAKE + 64), BAD), (dict(wsb=1000), BAD), (dict(B=4097), UNSUP), (dict(Hq=34), UNSUP),
    (dict(D=96), UNSUP), (dict(BS=8), UNSUP), (dict(NB=1 << 30), BAD), (dict(B=0), OK),
]


@pytest.mark.parametrize("over,status", COMMON + [(dict(window=0), BAD), (dict(window=-4), BAD),
                                                  (dict(dtype=F32, Hq=6), UNSUP)])
def test_decode_split_sinks_refuses(over, status):
    assert call("pa_decode_split_sinks", DECODE, over, SINKS_ORDER) == status


@pytest.mark.parametrize("over,status", COMMON + [(dict(window=-1), BAD), (dict(dtype=F32), UNSUP)])
def test_decode_q4_refuses(over, status):
    assert call("pa_decode_q4", DECODE, over, Q4_ORDER) == status


ROPE = dict(q=FAKE, k=FAKE + (1 << 20), v=FAKE + (1 << 21), qs=1024, ks=256, vs=256, pos=FAKE, inv=FAKE, slots=FAKE,
            T=4, Hq=8, Hkv=2, D=128, rd=128, inter=0, m=1.0, BS=16, NB=64, dtype=BF16,
            q_out=FAKE + (1 << 22), kp=FAKE, vp=FAKE, err=None, stream=None)
ROPE_ORDER = "q k v qs ks vs pos inv slots T Hq Hkv D rd inter m BS NB dtype q_out kp vp err stream".split()


@pytest.mark.parametrize("over,status", [
    (dict(T=-1), BAD), (dict(Hkv=0), BAD), (dict(NB=0), BAD), (dict(dtype=9), BAD), (dict(D=80), UNSUP),
    (dict(BS=64), UNSUP), (dict(rd=130), BAD), (dict(rd=-2), BAD), (dict(rd=15), BAD), (dict(rd=24), UNSUP),
    (dict(m=float("nan")), BAD), (dict(k=None), BAD), (dict(slots=None), BAD), (dict(pos=None), BAD),
    (dict(inv=None), BAD), (dict(q_out=None), BAD), (dict(qs=1020), BAD), (dict(ks=255), BAD), (dict(vs=260), BAD),
    (dict(q=FAKE + 8), BAD), (dict(kp=FAKE + 8), BAD), (dict(Hq=1 << 28, qs=1 << 40), UNSUP),
    (dict(q_out=FAKE + 16), BAD), (dict(q_out=FAKE + (1 << 20)), BAD), (dict(q_out=FAKE, qs=2048), BAD),
    (dict(q_out=FAKE + (1 << 21) - 16), BAD), (dict(T=0), OK),
])
@pytest.mark.parametrize("name", ["pa_rope_append", "pa_rope_append_q4"])
def test_rope_append_refuses(name, over, status):
    assert call(name, ROPE, over, ROPE_ORDER) == status


def test_the_4bit_calls_take_bf16_rows_only():
    assert call("pa_rope_append_q4", ROPE, dict(dtype=F32, qs=1024), ROPE_ORDER) == UNSUP
    lib = binding.library()
    assert lib.pa_kv_append_q4(FAKE, FAKE, 256, 256, FAKE, 4, 2, 128, 16, 8, F32, FAKE, FAKE, None, None) == UNSUP


def test_q4_append_and_gather_refuse():
    lib = binding.library()

    def append(k=FAKE, ks=256, slots=FAKE, T=4, H=2, D=128, BS=16, NB=8, kp=FAKE):
        return lib.pa_kv_append_q4(k, FAKE, ks, 256, slots, T, H, D, BS, NB, BF16, kp, FAKE, None, None)
    assert append(k=None) == append(slots=None) == append(ks=128) == append(ks=257) == BAD
    assert append(T=-1) == append(H=0) == append(NB=0) == append(kp=FAKE + 2) == BAD
    assert append(D=32) == append(BS=48) == UNSUP and append(T=0) == OK

    def gather(k=FAKE, slots=FAKE, T=4, H=2, D=128, BS=16, NB=8, dt=BF16, out=FAKE):
        return lib.pa_kv_gather_q4(k, FAKE, slots, T, H, D, BS, NB, dt, out, FAKE, None, None)
    assert gather(k=None) == gather(slots=None) == gather(T=-2) == gather(H=0) == gather(dt=3) == BAD
    assert gather(out=FAKE + 8) == BAD and gather(D=48) == gather(BS=24) == UNSUP and gather(T=0) == OK


EXTEND = dict(bt=FAKE, ctx=FAKE + (1 << 16), new=FAKE + (2 << 16), B=4, MBS=8, BS=16, queue=FAKE + (3 << 16), NB=64,
              state=FAKE + (4 << 16), T=100, ctx_out=FAKE + (5 << 16), qs=FAKE + (6 << 16), pos=FAKE + (7 << 16),
              slots=FAKE + (8 << 16), so=FAKE + (9 << 16), err=None, stream=None)
EXTEND_ORDER = "bt ctx new B MBS BS queue NB state T ctx_out qs pos slots so err stream".split()


@pytest.mark.parametrize("over,status", [
    (dict(B=-1), BAD), (dict(T=-1), BAD), (dict(B=4097), UNSUP), (dict(MBS=0), BAD), (dict(BS=0), BAD),
    (dict(NB=0), BAD), (dict(MBS=1 << 27), BAD), (dict(queue=None), BAD), (dict(state=None), BAD),
    (dict(ctx=None), BAD), (dict(bt=None), BAD), (dict(ctx_out=None), BAD), (dict(qs=None), BAD),
    (dict(slots=None), BAD), (dict(pos=FAKE + (7 << 16) + 4), BAD), (dict(slots=FAKE + 8), BAD),
    (dict(ctx_out=FAKE + (1 << 16)), BAD), (dict(so=FAKE + (4 << 16) + 4), BAD), (dict(qs=FAKE + 16), BAD),
    (dict(pos=FAKE + (8 << 16) + 16), BAD), (dict(queue=FAKE + 4), BAD),
])
def test_extend_tables_refuses(over, status):
    assert call("pa_extend_tables", EXTEND, over, EXTEND_ORDER) == status


def test_tile_bytes():
    lib = binding.library()
    assert lib.pa_q4_tile_bytes(16, 128) == 16 * 64 + 16 * 2 * 4
    assert lib.pa_q4_tile_bytes(32, 64) == 32 * 32 + 32 * 4 and lib.pa_q4_tile_bytes(16, 256) == 2304
    assert lib.pa_q4_tile_bytes(16, 96) == lib.pa_q4_tile_bytes(8, 64) == 0
    with pytest.raises(PagedKVError):
        binding.q4_tile_bytes(16, 96)


@pytest.mark.parametrize("rd", [16, 64, 128])
@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 4.0), ("ntk", 8.0), ("yarn", 16.0),
                                            ("yarn", 1.0)])
def test_rope_frequencies(rd, scaling, factor):
    inv, m = binding.rope_frequencies(rd, 10000.0, scaling, factor, device="cpu")
    i = np.arange(rd // 2)
    plain = 10000.0 ** (-2.0 * i / rd)
    if scaling == "none":
        want = plain
    elif scaling == "linear":
        want = plain / factor
    elif scaling == "ntk":
        # the last pair turns `factor` times more slowly, the first as before
        want = plain * factor ** (-2.0 * i / (rd - 2))
        assert math.isclose(want[-1], plain[-1] / factor)
    else:
        # pairs of more than 32 turns over 4096 tokens are kept, of less than one divided
        turns = 4096 * plain / (2 * math.pi)
        want = inv.numpy().astype(float)
        keep, cut = turns > 32, turns < 1
        # (the ramp's ends are whole pair numbers: one pair on either side may lie on it)
        np.testing.assert_allclose(want[:max(0, keep.sum() - 1)], plain[:max(0, keep.sum() - 1)], rtol=1e-6)
        if cut.sum() > 1:
            np.testing.assert_allclose(want[-(cut.sum() - 1):], plain[-(cut.sum() - 1):] / factor, rtol=1e-6)
        assert np.all(want <= plain * (1 + 1e-6)) and np.all(want >= plain / factor * (1 - 1e-6))
        assert math.isclose(m, 0.1 * math.log(factor) + 1, rel_tol=1e-6)
    np.testing.assert_allclose(inv.numpy(), want, rtol=2.0 ** -23)
    if scaling != "yarn":
        assert m == 1.0


@pytest.mark.parametrize("over", [dict(rotary_dim=0), dict(rotary_dim=7), dict(base=1.0), dict(base=float("nan")),
                                  dict(scaling="bend"), dict(scaling="ntk", factor=0.5),
                                  dict(scaling="ntk", rotary_dim=2), dict(scaling="yarn", original_context=0),
                                  dict(scaling="yarn", beta_fast=1.0, beta_slow=2.0),
                                  dict(scaling="linear", factor=float("inf"))])
def test_rope_frequencies_refuses(over):
    with pytest.raises(InvalidArgumentError):
        binding.rope_frequencies(**{"rotary_dim": 64, "factor": 2.0, "device": "cpu", **over})


def test_python_layer_refuses_host_tensors_and_shapes():
    bf = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    pool = torch.zeros(4, 2, binding.q4_tile_bytes(16, 64), dtype=torch.uint8)
    slots = torch.zeros(3, dtype=torch.int64)
    i32 = torch.zeros(3, dtype=torch.int32)
    for fn in (lambda: binding.kv_append_q4(bf, bf, slots, pool, pool),
               lambda: binding.kv_gather_q4(pool, pool, slots, 64),
               lambda: binding.kv_gather_q4(pool, pool[:2], slots, 64),
               lambda: binding.kv_gather_q4(pool[:, :, :-1], pool[:, :, :-1], slots, 64),
               lambda: binding.decode_q4(bf, pool, pool, i32[:, None], i32, 0.1),
               lambda: binding.decode_split_sinks(bf, pool, pool, i32[:, None], i32, 0.1, 4, 1),
               lambda: binding.rope_append(None, bf, bf, i32, torch.zeros(32), slots, pool, pool),
               lambda: binding.extend_tables(i32[:, None], i32, i32, i32, i32[:2], 16, 3,
                                             out=binding.StepTables.empty(3, 3, "cpu"))):
        with pytest.raises(InvalidArgumentError):
            fn()


def test_entry_points_open_ranges_and_reject_with_text():
    import os
    from paged_kv_cache_336_b200 import build
    for name, path in (("pa_decode_split_sinks", "decode_api.cu"), ("pa_decode_q4", "decode_api.cu"),
                       ("pa_rope_append", "rope_append.cu"), ("pa_rope_append_q4", "rope_append.cu"),
                       ("pa_kv_append_q4", "rope_append.cu"), ("pa_kv_gather_q4", "rope_append.cu"),
                       ("pa_extend_tables", "extend_tables.cu")):
        assert f'PA_NVTX_RANGE("{name}");' in open(os.path.join(build.CSRC, path)).read(), name
    assert call("pa_decode_q4", DECODE, dict(window=-1), Q4_ORDER) == BAD
    assert b"window" in binding.library().pa_last_error_string()
    m = ctypes.c_float()
    assert binding.library().pa_rope_frequencies(64, 1e4, 9, 2.0, 1, 2.0, 1.0, FAKE, ctypes.byref(m)) == BAD
