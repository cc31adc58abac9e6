"""pa_decode_split_sinks against the oracle's visible-token definition: sinks
that end before, inside and past the window, released blocks, fp32 and bf16,
every head_dim, few and many pieces."""

import numpy as np
import pytest
import torch

import oracle
from paged_kv_cache_336_b200 import binding, workloads

from gpu_util import check_close, device_tables, setup, to_f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,G,bs,D", [
    (workloads.F32, 1, 16, 128), (workloads.F32, 2, 32, 64), (workloads.F32, 8, 16, 64),
    (workloads.F32, 4, 32, 128), (workloads.BF16, 1, 32, 128),
    (workloads.BF16, 8, 16, 128), (workloads.BF16, 6, 16, 64), (workloads.BF16, 16, 32, 256)])
@pytest.mark.parametrize("window,sinks", [(1, 1), (7, 4), (40, 16), (40, 17), (16, 37), (97, 0),
                                          (33, 150), (30, 5000), (10_000, 4)])
def test_matches_oracle(dtype, G, bs, D, window, sinks):
    w = workloads.random_small(40 + G + bs, num_seqs=8, num_q_heads=2 * G, num_kv_heads=2,
                               head_dim=D, block_size=bs, dtype=dtype, max_ctx=12 * bs,
                               fixed_lens=[0, 1, 12 * bs, bs + 1, window + 1 if window < 150 else 2])
    bm, k_pool, v_pool = setup(w)
    q = workloads.draw_queries(w, 8, device="cuda")
    bt, ctx, tables, ctx_np = device_tables(bm, list(range(8)))
    want = oracle.paged_decode_sinks(to_f64(q), to_f64(k_pool), to_f64(v_pool), tables, ctx_np,
                                     w.scale, window, sinks)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = binding.decode_split_sinks(q, k_pool, v_pool, bt, ctx, w.scale, window, sinks,
                                     partition_tokens=2 * bs, dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    check_close(to_f64(out), want, dtype, f"window {window} sinks {sinks}")
    # blocks that hold neither a sink nor a token of the window are never read
    hidden = bt.clone()
    for s in range(8):
        for b in range(bt.shape[1]):
            t = np.arange(b * bs, min((b + 1) * bs, int(ctx_np[s])))
            if not ((t >= int(ctx_np[s]) - window) | (t < sinks)).any():
                hidden[s, b] = -1
    again = binding.decode_split_sinks(q, k_pool, v_pool, hidden, ctx, w.scale, window, sinks,
                                       partition_tokens=2 * bs, dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and torch.equal(out, again)
    if sinks == 0:
        ref = binding.decode_split_window(q, k_pool, v_pool, bt, ctx, w.scale, window, partition_tokens=2 * bs)
        check_close(to_f64(ref), to_f64(out), dtype, "no sinks is the window")


def test_rows_outside_what_is_visible_may_hold_anything():
    """NaN everywhere but in the visible tokens."""
    bs, window, sinks = 16, 21, 5
    w = workloads.random_small(77, num_seqs=4, num_q_heads=8, num_kv_heads=2, head_dim=128,
                               block_size=bs, dtype=workloads.BF16, max_ctx=200,
                               fixed_lens=[200, 31, 22, 100])
    bm, k_pool, v_pool = setup(w)
    q = workloads.draw_queries(w, 4, device="cuda")
    bt, ctx, tables, ctx_np = device_tables(bm, list(range(4)))
    want = binding.decode_split_sinks(q, k_pool, v_pool, bt, ctx, w.scale, window, sinks)
    see = torch.zeros(k_pool.shape[0], bs, dtype=torch.bool)
    for s in range(4):
        for t in range(int(ctx_np[s])):
            if t >= int(ctx_np[s]) - window or t < sinks:
                see[int(tables[s, t // bs]), t % bs] = True
    hide = ~see.cuda()[:, None, :, None].expand_as(k_pool)
    k_pool[hide] = float("nan")
    v_pool[hide] = float("nan")
    got = binding.decode_split_sinks(q, k_pool, v_pool, bt, ctx, w.scale, window, sinks)
    assert torch.equal(got, want)


def test_long_contexts_many_pieces():
    w = workloads.random_small(6, num_seqs=3, num_q_heads=8, num_kv_heads=2, head_dim=128,
                               block_size=16, dtype=workloads.BF16, max_ctx=40000,
                               fixed_lens=[40000, 33333, 900])
    bm, k_pool, v_pool = setup(w)
    q = workloads.draw_queries(w, 3, device="cuda")
    bt, ctx, tables, ctx_np = device_tables(bm, [0, 1, 2])
    want = oracle.paged_decode_sinks(to_f64(q), to_f64(k_pool), to_f64(v_pool), tables, ctx_np,
                                     w.scale, 9000, 1000)
    got = binding.decode_split_sinks(q, k_pool, v_pool, bt, ctx, w.scale, 9000, 1000)
    check_close(to_f64(got), want, workloads.BF16, "long")


def test_fp32_groups_cut_or_whole():
    """A group of 8 fp32 heads: few sequences (its heads dealt to several warps)
    and the same ones inside a large batch (where they stay together)."""
    w = workloads.random_small(31, num_seqs=400, num_q_heads=16, num_kv_heads=2, head_dim=64,
                               block_size=16, dtype=workloads.F32, max_ctx=100,
                               fixed_lens=[100, 64, 99])
    bm, k_pool, v_pool = setup(w)
    q = workloads.draw_queries(w, 400, device="cuda")
    bt, ctx, tables, ctx_np = device_tables(bm, list(range(400)))
    many = binding.decode_split_sinks(q, k_pool, v_pool, bt, ctx, w.scale, 40, 3)
    few = binding.decode_split_sinks(q[:3], k_pool, v_pool, bt[:3], ctx[:3], w.scale, 40, 3)
    want = oracle.paged_decode_sinks(to_f64(q[:3]), to_f64(k_pool), to_f64(v_pool), tables[:3], ctx_np[:3],
                                     w.scale, 40, 3)
    check_close(to_f64(few), want, workloads.F32, "few")
    check_close(to_f64(many[:3]), want, workloads.F32, "many")


@pytest.mark.parametrize("dtype", [workloads.F32, workloads.BF16])
def test_bad_blocks_give_zeros_and_spare_the_neighbour(dtype):
    w = workloads.random_small(91, num_seqs=2, num_q_heads=4, num_kv_heads=2, head_dim=64, block_size=16,
                               dtype=dtype, max_ctx=900, fixed_lens=[900, 70])
    bm, k_pool, v_pool = setup(w)
    q = workloads.draw_queries(w, 2, device="cuda")
    bt, ctx, _, _ = device_tables(bm, [0, 1])
    want = binding.decode_split_sinks(q, k_pool, v_pool, bt, ctx, w.scale, 500, 20, partition_tokens=16)
    bt[0] = 10 ** 6
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = binding.decode_split_sinks(q, k_pool, v_pool, bt, ctx, w.scale, 500, 20, partition_tokens=16, dev_err=err)
    assert int(err.item()) == binding.DEVERR_BLOCK_ID
    assert torch.all(got[0] == 0) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", [workloads.F32, workloads.BF16])
def test_many_sequences(dtype):
    w = workloads.random_small(92, num_seqs=4096, num_q_heads=1, num_kv_heads=1, head_dim=64, block_size=16,
                               dtype=dtype, max_ctx=40, fixed_lens=[0, 40, 33])
    bm, k_pool, v_pool = setup(w)
    q = workloads.draw_queries(w, 4096, device="cuda")
    bt, ctx, tables, ctx_np = device_tables(bm, list(range(4096)))
    want = oracle.paged_decode_sinks(to_f64(q), to_f64(k_pool), to_f64(v_pool), tables, ctx_np, w.scale, 9, 3)
    got = binding.decode_split_sinks(q, k_pool, v_pool, bt, ctx, w.scale, 9, 3)
    check_close(to_f64(got), want, dtype, "4096 sequences")


def test_host_validation_looks_at_visible_blocks_only():
    """PAGEDKV_VALIDATE=1 (read once per process): tables with released blocks pass
    a windowed call, a bad visible block is refused."""
    import os
    import subprocess
    import sys
    code = """
import torch
from paged_kv_cache_336_b200 import binding
q = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="cuda")
k, v = binding.q4_pools(8, 1, 16, 64)
t = torch.tensor([[0, -1, -1, 2, 3]], dtype=torch.int32, device="cuda")
c = torch.tensor([70], dtype=torch.int32, device="cuda")
kk = torch.zeros(8, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
binding.decode_q4(q, k, v, t, c, 0.1, window=20, sinks=3)
binding.decode_split_sinks(q, kk, kk, t, c, 0.1, 20, 3)
for f in (lambda: binding.decode_q4(q, k, v, t, c, 0.1), lambda: binding.decode_split_sinks(q, kk, kk, t, c, 0.1, 40, 3)):
    try:
        f()
    except binding.InvalidArgumentError:
        continue
    raise SystemExit("a bad block was accepted")
torch.cuda.synchronize()
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], env={**os.environ, "PAGEDKV_VALIDATE": "1", "PYTHONPATH": root},
                       cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("num", [1, 9, 900])
def test_short_windows_whole_and_cut(num):
    """Windows of a few units: one warp a sequence while a wave of CTAs holds
    them, an equal cut beyond."""
    w = workloads.random_small(95 + num, num_seqs=num, num_q_heads=16, num_kv_heads=4, head_dim=64, block_size=16,
                               dtype=workloads.BF16, max_ctx=130, fixed_lens=[130, 60, 61][:num])
    bm, k_pool, v_pool = setup(w)
    q = workloads.draw_queries(w, num, device="cuda")
    bt, ctx, tables, ctx_np = device_tables(bm, list(range(num)))
    want = oracle.paged_decode_sinks(to_f64(q), to_f64(k_pool), to_f64(v_pool), tables, ctx_np, w.scale, 50, 9)
    got = binding.decode_split_sinks(q, k_pool, v_pool, bt, ctx, w.scale, 50, 9)
    check_close(to_f64(got), want, workloads.BF16, "short windows")


@pytest.mark.parametrize("dtype,Hq", [(workloads.F32, 8), (workloads.BF16, 12)])
@pytest.mark.parametrize("window,sinks", [(700, 4), (33, 0), (20, 700), (5000, 1)])
@pytest.mark.parametrize("partition_tokens", [512, 1024])
def test_sequences_cut_one_by_one(dtype, Hq, window, sinks, partition_tokens):
    """Tables of up to three partitions: each sequence is cut by itself into equal
    pieces, some of them empty for short sequences."""
    w = workloads.random_small(97, num_seqs=6, num_q_heads=Hq, num_kv_heads=2, head_dim=64, block_size=32,
                               dtype=dtype, max_ctx=1400, fixed_lens=[1400, 0, 1, 17, 70, 1399])
    bm, k_pool, v_pool = setup(w)
    q = workloads.draw_queries(w, 6, device="cuda")
    bt, ctx, tables, ctx_np = device_tables(bm, list(range(6)))
    want = oracle.paged_decode_sinks(to_f64(q), to_f64(k_pool), to_f64(v_pool), tables, ctx_np, w.scale, window, sinks)
    got = binding.decode_split_sinks(q, k_pool, v_pool, bt, ctx, w.scale, window, sinks,
                                     partition_tokens=partition_tokens)
    check_close(to_f64(got), want, dtype, "cut one by one")
