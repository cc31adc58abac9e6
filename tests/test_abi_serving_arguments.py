"""Arguments of the serving-step calls at the Python boundary: windows beyond 32
bits, tensors of other ranks. Stand-ins for device tensors and for the library, which records its call."""

import pytest
import torch

from paged_kv_cache_336_b200 import binding

from test_abi_serving_devices import CALLS, OnDevice, workspace


@pytest.fixture
def made(monkeypatch):
    """The (name, arguments) of the calls that reached the library."""
    calls = []

    class Library:
        def __getattr__(self, name):
            def record(*args):
                calls.append((name, args))
                return binding.PA_OK
            return record
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(binding, "_stream_ptr", lambda stream: 0)
    monkeypatch.setattr(binding, "library", Library)
    return calls


def tensors(name):
    return {k: OnDevice(*a) for k, a in CALLS[name][0].items()}


@pytest.mark.parametrize("given,passed", [(5, 5), (0x7fffffff, 0x7fffffff), (1 << 31, 0x7fffffff),
                                          ((1 << 32) + 5, 0x7fffffff), (1 << 70, 0x7fffffff), (-1, -1), (-3, -1),
                                          (-(1 << 32) + 5, -1)])
def test_windows_and_sinks_do_not_wrap(made, given, passed):
    x = tensors("sinks")
    binding.decode_split_sinks(x["q"], x["k"], x["v"], x["bt"], x["ctx"], 0.1, given, given, out=x["out"],
                               workspace=workspace(0))
    assert made.pop()[1][15:17] == (passed, passed)
    x = tensors("q4")
    binding.decode_q4(x["q"], x["k"], x["v"], x["bt"], x["ctx"], 0.1, window=given, sinks=given, out=x["out"],
                      workspace=workspace(0))
    assert made.pop()[1][14:16] == (passed, passed)


RANKED = [("sinks", "q"), ("sinks", "k"), ("sinks", "bt"), ("sinks", "ctx"), ("q4", "q"), ("q4", "k"), ("q4", "bt"),
          ("q4", "ctx"), ("append", "k"), ("append", "v"), ("append", "slots"), ("append", "kp"), ("gather", "kp"),
          ("gather", "slots"), ("gather", "ko"), ("rope", "q"), ("rope", "k"), ("rope", "v"), ("rope", "kp"),
          ("rope", "pos"), ("rope", "slots"), ("rope", "inv"), ("rope", "qo"), ("extend", "bt")]


@pytest.mark.parametrize("name,which", RANKED)
@pytest.mark.parametrize("more", [True, False])
def test_a_tensor_of_another_rank_is_refused(made, name, which, more):
    """With the package's own error, one dimension too many or too few."""
    args, call = CALLS[name]
    shape, dtype = args[which]
    x = {**tensors(name), which: OnDevice((*shape, 1) if more else shape[1:], dtype)}
    with pytest.raises(binding.InvalidArgumentError):
        call(x, workspace(0))
    assert not made


@pytest.mark.parametrize("head_dim", [0, -64, 48])
def test_a_head_dim_that_the_tiles_do_not_hold(made, head_dim):
    x = tensors("gather")
    with pytest.raises(binding.InvalidArgumentError):
        binding.kv_gather_q4(x["kp"], x["vp"], x["slots"], head_dim)
    assert not made
