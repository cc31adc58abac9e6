"""Outputs that share memory with what the same call reads or writes are refused
(CPU: the checks come before any device call). Sizes are those of each array, so
neighbours in one allocation pass the check."""

import pytest

from paged_kv_cache_336_b200 import binding

BAD, CUDA = binding.PA_ERR_INVALID_ARG, binding.PA_ERR_CUDA
MIB = 1 << 20
BASE = 0x7000_0000
T, HQ, HKV, D, BS, NB = 64, 8, 2, 128, 16, 32
Q_BYTES = T * HQ * D * 2
POOL16, POOL4 = NB * HKV * BS * D * 2, NB * HKV * 9 * D

ROPE_ORDER = "q k v qs ks vs pos inv slots T Hq Hkv D rd inter m BS NB dtype q_out kp vp err stream".split()
ROPE = dict(q=BASE, k=BASE + 16 * MIB, v=BASE + 17 * MIB, qs=HQ * D, ks=HKV * D, vs=HKV * D, pos=BASE + 18 * MIB,
            inv=BASE + 19 * MIB, slots=BASE + 20 * MIB, T=T, Hq=HQ, Hkv=HKV, D=D, rd=D, inter=0, m=1.0, BS=BS, NB=NB,
            dtype=binding.PA_BF16, q_out=BASE + 32 * MIB, kp=BASE + 48 * MIB, vp=BASE + 64 * MIB, err=None, stream=None)


def no_launch():
    import torch
    return not torch.cuda.is_available()


def rope(name, **over):
    a = {**ROPE, **over}
    return getattr(binding.library(), name)(*[a[k] for k in ROPE_ORDER])


@pytest.mark.parametrize("name,pool", [("pa_rope_append", POOL16), ("pa_rope_append_q4", POOL4)])
def test_q_out_overlaps_nothing(name, pool):
    for key, size in (("kp", pool), ("vp", pool), ("pos", T * 4), ("slots", T * 8), ("inv", D * 2)):
        assert rope(name, **{key: ROPE["q_out"]}) == BAD, key
        assert rope(name, **{key: ROPE["q_out"] + Q_BYTES - 16}) == BAD, key
        assert rope(name, **{key: ROPE["q_out"] - size + 16}) == BAD, key
    # what is not read may stand anywhere: no rotation, no queries
    if no_launch():  # (without a device the accepted call ends in the launch's error)
        assert rope(name, rd=0, pos=ROPE["q_out"], inv=ROPE["q_out"]) == CUDA
        assert rope(name, kp=ROPE["q_out"] - pool, vp=ROPE["q_out"] + Q_BYTES) == CUDA
        assert rope(name, q_out=ROPE["q"]) == CUDA


def test_the_4bit_read_overlaps_nothing():
    rows = T * HKV * D * 2

    def gather(ko=BASE + 32 * MIB, vo=BASE + 40 * MIB, kp=BASE, vp=BASE + 8 * MIB, slots=BASE + 16 * MIB):
        return binding.library().pa_kv_gather_q4(kp, vp, slots, T, HKV, D, BS, NB, binding.PA_BF16, ko, vo, None, None)

    assert gather(vo=BASE + 32 * MIB) == BAD and gather(vo=BASE + 32 * MIB + rows - 16) == BAD
    for key, size in (("kp", POOL4), ("vp", POOL4), ("slots", T * 8)):
        for out in (BASE + 32 * MIB, BASE + 40 * MIB):
            assert gather(**{key: out + rows - 16}) == BAD and gather(**{key: out - size + 16}) == BAD
    if no_launch():
        assert gather(vo=BASE + 32 * MIB + rows, kp=BASE + 32 * MIB - POOL4) == CUDA
