"""pa_extend_tables at batch sizes whose shared memory lies around what a kernel
gets without opting in, each in a process of its own."""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu


FRESH = """
import sys
import torch
from paged_kv_cache_336_b200 import binding
n = int(sys.argv[1])
i32 = dict(dtype=torch.int32, device="cuda")
tables = torch.full((n, 2), -1, **i32)
queue = torch.arange(n, **i32)
out = binding.extend_tables(tables, torch.zeros(n, **i32), torch.ones(n, **i32), queue,
                            torch.tensor([0, n], **i32), 16, n)
torch.cuda.synchronize()
assert torch.equal(tables[:, 0], queue) and torch.all(tables[:, 1] == -1)
assert torch.equal(out.slot_mapping, 16 * torch.arange(n, device="cuda"))
assert torch.equal(out.query_start, torch.arange(n + 1, **i32)) and out.queue_state.tolist() == [0, 0]
"""


@pytest.mark.parametrize("num", [3000, 3008, 3058, 3059, 3071, 3072, 4096])
def test_every_batch_size_runs_in_a_fresh_process(num):
    """Around 48 KB of shared memory, with no earlier call of a larger batch."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FRESH, str(num)], env={**os.environ, "PYTHONPATH": root},
                       cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
