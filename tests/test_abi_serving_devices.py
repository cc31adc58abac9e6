"""The serving-step calls refuse tensors, workspaces and error words that are not
on the current device: a kernel there would touch memory that it may not reach.
Stand-ins for device tensors, so that no GPU is needed and none is reached."""

import pytest
import torch

from paged_kv_cache_336_b200 import binding
from paged_kv_cache_336_b200.binding import InvalidArgumentError

I32, I64, BF16, U8 = torch.int32, torch.int64, torch.bfloat16, torch.uint8


class OnDevice:
    """What the binding asks of a device tensor; `device` -1 is the host."""

    def __init__(self, shape, dtype, device=0):
        self._like = torch.empty(shape, dtype=dtype, device="meta")
        self._device = device
        self.is_cuda = device >= 0
        self.dtype, self.shape = dtype, self._like.shape

    def get_device(self):
        return self._device

    def data_ptr(self):
        return 0x7000_0000

    def __getattr__(self, name):  # is_contiguous, dim, numel, size, stride, element_size
        return getattr(self._like, name)


@pytest.fixture(autouse=True)
def device_zero_is_current(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(binding, "_stream_ptr", lambda stream: 0)

    class NoLibrary:
        def __getattr__(self, name):
            def reached(*args):
                raise AssertionError(f"{name} was reached")
            return reached
    monkeypatch.setattr(binding, "library", NoLibrary)


def workspace(device):
    ws = binding.SplitWorkspace.__new__(binding.SplitWorkspace)
    ws.device, ws.ptr, ws.nbytes, ws.partition_tokens = device, 1 << 20, 1 << 20, 64
    return ws


B, HQ, HKV, D, BS, MBS, NB, T = 2, 4, 2, 64, 16, 3, 8, 5
TILE = 9 * D


def decode_args(pool):
    return dict(q=((B, HQ, D), BF16), k=(pool, BF16 if len(pool) == 4 else U8), v=(pool, BF16 if len(pool) == 4 else U8),
                bt=((B, MBS), I32), ctx=((B,), I32), out=((B, HQ, D), BF16), err=((1,), I32))


CALLS = {
    "sinks": (decode_args((NB, HKV, BS, D)), lambda x, ws: binding.decode_split_sinks(
        x["q"], x["k"], x["v"], x["bt"], x["ctx"], 0.1, 32, 4, out=x["out"], workspace=ws, dev_err=x["err"])),
    "q4": (decode_args((NB, HKV, TILE)), lambda x, ws: binding.decode_q4(
        x["q"], x["k"], x["v"], x["bt"], x["ctx"], 0.1, out=x["out"], workspace=ws, dev_err=x["err"])),
    "append": (dict(k=((T, HKV, D), BF16), v=((T, HKV, D), BF16), slots=((T,), I64), kp=((NB, HKV, TILE), U8),
                    vp=((NB, HKV, TILE), U8), err=((1,), I32)),
               lambda x, ws: binding.kv_append_q4(x["k"], x["v"], x["slots"], x["kp"], x["vp"], dev_err=x["err"])),
    "gather": (dict(kp=((NB, HKV, TILE), U8), vp=((NB, HKV, TILE), U8), slots=((T,), I64), ko=((T, HKV, D), BF16),
                    vo=((T, HKV, D), BF16), err=((1,), I32)),
               lambda x, ws: binding.kv_gather_q4(x["kp"], x["vp"], x["slots"], D, out=(x["ko"], x["vo"]),
                                                  dev_err=x["err"])),
    "rope": (dict(q=((T, HQ, D), BF16), k=((T, HKV, D), BF16), v=((T, HKV, D), BF16), pos=((T,), I32),
                  inv=((D // 2,), torch.float32), slots=((T,), I64), kp=((NB, HKV, BS, D), BF16),
                  vp=((NB, HKV, BS, D), BF16), qo=((T, HQ, D), BF16), err=((1,), I32)),
             lambda x, ws: binding.rope_append(x["q"], x["k"], x["v"], x["pos"], x["inv"], x["slots"], x["kp"],
                                               x["vp"], q_out=x["qo"], dev_err=x["err"])),
    "extend": (dict(bt=((B, MBS), I32), ctx=((B,), I32), new=((B,), I32), queue=((NB,), I32), state=((2,), I32),
                    o1=((B,), I32), o2=((B + 1,), I32), o3=((T,), I32), o4=((T,), I64), o5=((2,), I32), err=((1,), I32)),
               lambda x, ws: binding.extend_tables(
                   x["bt"], x["ctx"], x["new"], x["queue"], x["state"], BS, T,
                   out=binding.StepTables(x["o1"], x["o2"], x["o3"], x["o4"], x["o5"]), dev_err=x["err"])),
}


@pytest.mark.parametrize("name,which", [(n, w) for n, (args, _) in CALLS.items() for w in list(args) + [None]])
def test_every_tensor_is_looked_at(name, which):
    args, call = CALLS[name]

    def made(device):
        return {k: OnDevice(*a, device=device if k == which else 0) for k, a in args.items()}
    if which is None:
        with pytest.raises(AssertionError, match="was reached"):  # nothing is wrong: the call is made
            call(made(0), workspace(0))
        return
    for device in (1, -1):
        with pytest.raises(InvalidArgumentError):
            call(made(device), workspace(0))


@pytest.mark.parametrize("name", ["sinks", "q4"])
def test_a_workspace_of_another_device_is_refused(name):
    args, call = CALLS[name]
    with pytest.raises(InvalidArgumentError):
        call({k: OnDevice(*a) for k, a in args.items()}, workspace(1))


def test_an_error_word_has_32_bits():
    args, call = CALLS["append"]
    for shape, dtype in (((1,), U8), ((1,), I64), ((0,), I32)):
        with pytest.raises(InvalidArgumentError):
            call({**{k: OnDevice(*a) for k, a in args.items()}, "err": OnDevice(shape, dtype)}, None)
