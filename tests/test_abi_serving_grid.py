"""The grids of the serving-step operators follow the device's multiprocessor
count, which one helper of the library asks for."""

import os
import re

import pytest

from paged_kv_cache_336_b200 import build


@pytest.mark.parametrize("name", ["extend_tables.cu", "rope_append.cu", "kv_ops.cu", "decode_q4_inst.cu",
                                  "decode_sinks_kernel.cuh"])
def test_no_multiprocessor_count_is_written_into_a_grid(name):
    text = open(os.path.join(build.CSRC, name)).read()
    code = re.sub(r"//[^\n]*", "", text)
    assert not re.search(r"\b148\b", code)
    if name in ("extend_tables.cu", "rope_append.cu", "kv_ops.cu"):
        assert "sm_count()" in code and "int sm_count()" not in code
